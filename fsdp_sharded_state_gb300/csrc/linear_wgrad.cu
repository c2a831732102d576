// linear_wgrad.cu -- dw (+)= dz^T x, the weight gradient of a linear layer, and db (+)= the
// column sums of dz.
#include "linear_launch.cuh"

namespace fsdp {

namespace {
// The sum of `parts` partial sums for each element of out ([parts][rows][ld], rows x cols of it)
// and then of db ([parts][rows]): a CTA takes 32 elements, warp w parts w, w + 8, .., and the
// warps' sums are added in order.  With a thread to an element the parts are as many latencies as
// they are groups of 16: wgrad of 16384 x 64 x 32 fp32 (64 parts) took 14.9 us instead of 6.3,
// 2048 x 64 x 64 (16 parts) 6.3 instead of 4.7.
template <typename OT>
__global__ void __launch_bounds__(256)
k_join(const float* __restrict__ part, const float* __restrict__ db_part, int parts, int64_t rows, int64_t cols, int64_t ld, OT* out,
       int64_t ldo, OT* db, int accumulate) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = int64_t(blockIdx.x) * 32 + lane, n = rows * cols;
    const bool is_db = i >= n, in = i < n + (db ? rows : 0);
    const int64_t r = is_db ? i - n : i / cols, c = is_db ? 0 : i - r * cols;
    const float* p = is_db ? db_part + r : part + r * ld + c;
    const int64_t step = is_db ? rows : rows * ld;
    pdl_wait();
    float t = 0.f;
#pragma unroll 8
    for (int s = warp; s < parts; s += 8) t += in ? p[s * step] : 0.f;
    sums[warp][lane] = t;
    __syncthreads();
    if (warp > 0 || !in) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) t += sums[w][lane];
    OT* const o = is_db ? db + r : out + r * ldo + c;
    store1(o, accumulate ? t + load1(o) : t);
}

template <typename OT>
cudaError_t join(const float* part, const float* db_part, int parts, int64_t rows, int64_t cols, int64_t ld, const LinEpi& ep,
                 cudaStream_t st) {
    const int64_t blocks = ceil_div(rows * cols + (ep.db ? rows : 0), 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch(k_join<OT>, dim3(unsigned(blocks)), dim3(256), 0, st, part, db_part, parts, rows, cols, ld,
                  static_cast<OT*>(ep.out), ep.ldo, static_cast<OT*>(ep.db), int(ep.accumulate));
}

template <typename OT, int PL, int CH>
cudaError_t launch_pair_wgrad(const LinProblem& p, int bn, cudaStream_t st) {
    if (CH == 0 && p.epi.vec != 2) return launch_pair_as<kWgrad, OT, PL, CH, -1, CH == 0>(p, bn, st);
    return launch_pair_as<kWgrad, OT, PL, CH>(p, bn, st);
}
}  // namespace

cudaError_t launch_linear_wgrad(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3)
        return p.out_bf16 ? launch_product<kWgrad, uint16_t, 3, 0>(p, launch_pair_wgrad<uint16_t, 3, 0>, st)
                          : launch_product<kWgrad, float, 3, 2>(p, launch_pair_wgrad<float, 3, 2>, st);
    return p.out_bf16 ? launch_product<kWgrad, uint16_t, 1, 0>(p, launch_pair_wgrad<uint16_t, 1, 0>, st)
                      : launch_product<kWgrad, float, 1, 8>(p, launch_pair_wgrad<float, 1, 8>, st);
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

cudaError_t launch_wgrad_slabs(const LinProblem& p, cudaStream_t st) {
    LinProblem q = p;
    const int64_t rows = p.epi.rows, cols = p.epi.cols, ld = (cols + 7) & ~int64_t(7);
    q.epi.out = p.partial;
    q.epi.ldo = ld;
    q.epi.db = p.epi.db ? p.partial + p.slabs * rows * ld : nullptr;
    q.epi.accumulate = 0;
    q.epi.vec = 1;
    cudaError_t e = p.planes == 3 ? launch_cfg<LinCfg<kWgrad, float, 1, 64, 3, 2, true>>(q, kSlabSplits, st, p.slabs)
                                  : launch_cfg<LinCfg<kWgrad, float, 1, 64, 1, 8, true>>(q, kSlabSplits, st, p.slabs);
    if (e != cudaSuccess) return e;
    const float* const db_part = p.partial + p.slabs * rows * ld;
    return launch_join(p.partial, db_part, p.slabs, rows, cols, ld, p.epi, p.out_bf16, st);
}

cudaError_t launch_join(const float* part, const float* db_part, int parts, int64_t rows, int64_t cols, int64_t ld, const LinEpi& ep,
                        bool out_bf16, cudaStream_t st) {
    return out_bf16 ? join<uint16_t>(part, db_part, parts, rows, cols, ld, ep, st)
                    : join<float>(part, db_part, parts, rows, cols, ld, ep, st);
}

cudaError_t take_wait_error_wgrad(unsigned int* flag) { return take_product_wait_error(flag); }

}  // namespace fsdp
