// norm_forward.cu -- y = (x - mean) * rstd * weight + bias, row by row.
//
// Bound by HBM: x read and y written once.  A row stays in registers; its mean is summed first
// and the squares of what is left after it, so that a common offset of the row costs no digits.
// What rounding did to that mean is taken out again: with d = x - mean, the sum of d is 0 but for
// it, and where d's own mean exceeds 2^-23 of d's root mean square, as in rows far from zero, the
// variance and y are formed from d less its mean.
#include "norm_rows.cuh"

namespace fsdp {
namespace {

struct ForwardArgs {
    const void* x;
    int64_t ldx;
    const void* weight;
    const void* bias;
    void* y;
    int64_t ldy;
    float* mean;
    float* rstd;
    int64_t rows;
    int32_t cols, ctas, stages, block;
    float eps;
    uint64_t wait_ns;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1024 / C::THREADS)
k_norm_forward(const __grid_constant__ ForwardArgs a) {
    using T = typename C::T;
    extern __shared__ __align__(128) unsigned char smem_raw[];   // the rings
    __shared__ __align__(16) float sums[C::GW > 1 ? 4 * kNormMaxWarps : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    RowRing<C, 1> ring = make_ring<C, 1>(smem_raw, warp, first, a.cols, a.stages, a.block, a.wait_ns);
    ring.base[0] = static_cast<const T*>(a.x) + first;
    ring.ld[0] = a.ldx;
    const bool issuer = C::GW == 1 || tid == 0;
    if (C::GW == 1 ? lane == 0 : tid == 0) ring.init();
    if constexpr (C::CLUSTER) {                  // no CTA writes to another that has not started
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    pdl_wait();
    // blocks of rows: a warp's (GW = 1), a CTA's or a cluster's (one row)
    const int64_t n_groups = int64_t(gridDim.x / a.ctas) * (C::GW == 1 ? 8 : 1), step = n_groups * a.block;
    const int64_t row0 = (blockIdx.x / a.ctas * (C::GW == 1 ? 8 : 1) + (C::GW == 1 ? warp : 0)) * int64_t(a.block);
    if (issuer) {
        for (int s = 0; s < a.stages; ++s)
            if (row0 + s * step < a.rows) ring.fetch(row0 + s * step, a.rows, s, lane);
    }
    float w[C::E], b[C::E];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
    norm_vector<C>(static_cast<const T*>(a.bias), a.cols, first, t, 0.f, b);
    RowSum<C, 2> sum{sums};
    const float n = float(a.cols);
    int s = 0;
    uint32_t phase = 0;
    auto next_stage = [&](int64_t row) {
        if (issuer && row + a.stages * step < a.rows) ring.fetch(row + a.stages * step, a.rows, s, lane);
        if (++s == a.stages) {
            s = 0;
            phase ^= 1;
        }
    };
    // the threads of a warp, CTA or cluster leave the loops together
    for (int64_t row = row0; row < a.rows; row += step) {
        ring.wait(s, phase);
        const int count = a.rows - row < a.block ? int(a.rows - row) : a.block;
        for (int j0 = 0; j0 < count; j0 += C::GW == 1 ? 32 / C::L : 1) {
            const int j = j0 + (C::GW == 1 ? lane / C::L : 0);
            const bool have = j < count;
            float x[C::E];
            if (have) {
                norm_load<C>(ring.row_of(row + j, j, s, 0) - first, a.cols, first, t, x);
            } else {
#pragma unroll
                for (int e = 0; e < C::E; ++e) x[e] = 0.f;
            }
            float v[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < C::E; ++e) v[0] += x[e];
            sum(v, warp, lane, a.ctas);
            if (C::GW > 1) next_stage(row);      // every thread has read the stage
            const float mean = v[0] / n;
            v[0] = v[1] = 0.f;
#pragma unroll
            for (int e = 0; e < C::E; ++e) {
                x[e] = norm_col<C>(first, t, e) < a.cols ? x[e] - mean : 0.f;
                v[0] += x[e];
                v[1] = __fmaf_rn(x[e], x[e], v[1]);
            }
            sum(v, warp, lane, a.ctas);
            // what the sum left of an offset far beyond the spread; below that it is the roundings
            // of the differences themselves, which need not average out
            float left = v[0] / n;
            if (left * left <= 1.5e-14f * (v[1] / n)) left = 0.f;
            float var = (v[1] - v[0] * left) / n;
            if (var < 0.f) var = 0.f;            // a NaN stays
            const float rstd = 1.f / sqrtf(var + a.eps);
            if (!have) continue;
#pragma unroll
            for (int e = 0; e < C::E; ++e) x[e] = __fmaf_rn((x[e] - left) * rstd, w[e], b[e]);
            norm_store<C>(static_cast<T*>(a.y) + (row + j) * a.ldy, a.cols, first, t, x);
            if (t == 0 && rank == 0) {
                if (a.mean) a.mean[row + j] = left == left ? mean + left : mean;   // an infinity stays
                if (a.rstd) a.rstd[row + j] = rstd;
            }
        }
        if (C::GW == 1) {
            __syncwarp();                        // every lane has read the stage
            next_stage(row);
        }
    }
    ring.leave();
}

template <class C>
cudaError_t launch_as(const NormProblem& p, cudaStream_t st) {
    static std::atomic<uint64_t> prepared{0};
    const int ctas = norm_ctas<C>(p.cols), per_sm = 1024 / C::THREADS;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = norm_prepare(k_norm_forward<C>, prepared, dev);
    if (e != cudaSuccess) return e;
    const RingShape ring = ring_shape<C>(1, p.cols, per_sm);
    const int64_t each = ring.block * (C::GW == 1 ? 8 : 1);
    const int64_t want = (p.rows + each - 1) / each, room = int64_t(norm_sms(dev)) * per_sm / ctas;
    const ForwardArgs a{p.x, p.ldx, p.weight, p.bias, p.y, p.ldy, p.mean, p.rstd, p.rows, int32_t(p.cols), ctas, ring.stages, ring.block,
                        p.eps, detail::kWaitNs};
    return norm_launch(k_norm_forward<C>, int(want < room ? want : room), ctas, C::THREADS, ring.bytes, st, a);
}

}  // namespace

cudaError_t launch_norm_forward(const NormProblem& p, cudaStream_t st) {
    auto go = [&](auto c) { return launch_as<decltype(c)>(p, st); };
    if (p.bf16) return p.vec ? norm_dispatch<uint16_t, true>(p.cols, go) : norm_dispatch<uint16_t, false>(p.cols, go);
    return p.vec ? norm_dispatch<float, true>(p.cols, go) : norm_dispatch<float, false>(p.cols, go);
}

cudaError_t take_wait_error_norm_forward(unsigned int* flag) { return take_norm_wait_error(flag); }

}  // namespace fsdp
