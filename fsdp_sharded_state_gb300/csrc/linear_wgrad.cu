// linear_wgrad.cu -- dw (+)= dz^T x, the weight gradient of a linear layer, and db (+)= the
// column sums of dz.
#include "linear_kernel.cuh"

namespace fsdp {

cudaError_t launch_linear_wgrad(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3)
        return p.out_bf16 ? launch_product<kWgrad, uint16_t, 3, 0>(p, launch_pair_as<kWgrad, uint16_t, 3, 0>, st)
                          : launch_product<kWgrad, float, 3, 2>(p, launch_pair_as<kWgrad, float, 3, 2>, st);
    return p.out_bf16 ? launch_product<kWgrad, uint16_t, 1, 0>(p, launch_pair_as<kWgrad, uint16_t, 1, 0>, st)
                      : launch_product<kWgrad, float, 1, 8>(p, launch_pair_as<kWgrad, float, 1, 8>, st);
}

// ---- slabs ------------------------------------------------------------------------------
// A small out leaves most SMs without a tile, even with 8 CTAs on each: then the rows are cut
// into slabs, each with partial sums of its own, added up in slab order by a second launch.
// The device holds 36 clusters of 4 such CTAs (15 of 8).
int wgrad_slabs(int64_t rows, int64_t in, int64_t out) {
    const int64_t tiles = ceil_div(out, 128) * ceil_div(in, 64), kb = ceil_div(rows, kKb);
    const int64_t by_room = 36 / tiles, by_rows = kb / (2 * kSlabSplits);   // at least two K steps for each CTA
    const int64_t s = by_room < by_rows ? by_room : by_rows;
    return s < 2 ? 0 : int(s);
}
int64_t wgrad_slab_floats(int64_t rows, int64_t in, int64_t out) {
    return int64_t(wgrad_slabs(rows, in, out)) * (out * ((in + 7) & ~int64_t(7)) + ((out + 3) & ~int64_t(3)));
}

namespace {
template <typename OT>
__global__ void __launch_bounds__(256)
k_join_slabs(const float* __restrict__ part, int slabs, int64_t rows, int64_t cols, int64_t ld, OT* out, int64_t ldo, OT* db,
             int accumulate) {
    pdl_wait();
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, n = rows * cols;
    const bool is_db = i >= n;
    if (i >= n + (db ? rows : 0)) return;
    const int64_t r = is_db ? i - n : i / cols, c = is_db ? 0 : i - r * cols;
    const float* p = is_db ? part + slabs * rows * ld + r : part + r * ld + c;
    const int64_t step = is_db ? rows : rows * ld;
    float t = p[0];
#pragma unroll 16
    for (int s = 1; s < slabs; ++s) t += p[s * step];
    OT* const o = is_db ? db + r : out + r * ldo + c;
    store1(o, accumulate ? t + load1(o) : t);
}
}  // namespace

cudaError_t launch_wgrad_slabs(const LinProblem& p, cudaStream_t st) {
    LinProblem q = p;
    const int64_t rows = p.epi.rows, cols = p.epi.cols, ld = (cols + 7) & ~int64_t(7);
    q.epi.out = p.partial;
    q.epi.ldo = ld;
    q.epi.db = p.epi.db ? p.partial + p.slabs * rows * ld : nullptr;
    q.epi.accumulate = 0;
    q.epi.vec = 2;
    cudaError_t e = p.planes == 3 ? launch_cfg<LinCfg<kWgrad, float, 1, 64, 3, 2, true>>(q, kSlabSplits, st, p.slabs)
                                  : launch_cfg<LinCfg<kWgrad, float, 1, 64, 1, 8, true>>(q, kSlabSplits, st, p.slabs);
    if (e != cudaSuccess) return e;
    const int64_t blocks = ceil_div(rows * cols + (p.epi.db ? rows : 0), 256);
    return p.out_bf16 ? launch(k_join_slabs<uint16_t>, dim3(unsigned(blocks)), dim3(256), 0, st, p.partial, p.slabs, rows, cols, ld,
                               static_cast<uint16_t*>(p.epi.out), p.epi.ldo, static_cast<uint16_t*>(p.epi.db), p.epi.accumulate)
                      : launch(k_join_slabs<float>, dim3(unsigned(blocks)), dim3(256), 0, st, p.partial, p.slabs, rows, cols, ld,
                               static_cast<float*>(p.epi.out), p.epi.ldo, static_cast<float*>(p.epi.db), p.epi.accumulate);
}

cudaError_t take_wait_error_wgrad(unsigned int* flag) { return take_local_wait_error(flag); }

}  // namespace fsdp
