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
    int32_t cols, ctas;
    float eps;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS)
k_norm_forward(const __grid_constant__ ForwardArgs a) {
    using T = typename C::T;
    __shared__ __align__(16) float sums[C::GW > 1 ? 4 * kNormMaxWarps : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    const int64_t step = int64_t(gridDim.x) / a.ctas * C::ROWS;
    int64_t row = int64_t(blockIdx.x) / a.ctas * C::ROWS + (C::GW == 1 ? tid / C::L : 0);
    if constexpr (C::CLUSTER) {                  // no CTA writes to another that has not started
        cluster_arrive();
        cluster_wait();
    }
    pdl_wait();
    float w[C::E], b[C::E];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
    norm_vector<C>(static_cast<const T*>(a.bias), a.cols, first, t, 0.f, b);
    RowSum<C, 2> sum{sums};
    const float n = float(a.cols);
    // the threads of a warp, CTA or cluster leave the loop together
    for (int64_t at = int64_t(blockIdx.x) / a.ctas * C::ROWS; at < a.rows; at += step, row += step) {
        const bool have = row < a.rows;
        float x[C::E];
        if (have) {
            norm_load<C>(static_cast<const T*>(a.x) + row * a.ldx, a.cols, first, t, x);
        } else {
#pragma unroll
            for (int e = 0; e < C::E; ++e) x[e] = 0.f;
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < C::E; ++e) s[0] += x[e];
        sum(s, warp, lane, a.ctas);
        const float mean = s[0] / n;
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            x[e] = norm_col<C>(first, t, e) < a.cols ? x[e] - mean : 0.f;
            s[0] += x[e];
            s[1] = __fmaf_rn(x[e], x[e], s[1]);
        }
        sum(s, warp, lane, a.ctas);
        // what the sum left of an offset far beyond the spread; below that it is the roundings
        // of the differences themselves, which need not average out
        float left = s[0] / n;
        if (left * left <= 1.5e-14f * (s[1] / n)) left = 0.f;
        float var = (s[1] - s[0] * left) / n;
        if (var < 0.f) var = 0.f;                // a NaN stays
        const float r = 1.f / sqrtf(var + a.eps);
        if (!have) continue;
#pragma unroll
        for (int e = 0; e < C::E; ++e) x[e] = __fmaf_rn((x[e] - left) * r, w[e], b[e]);
        norm_store<C>(static_cast<T*>(a.y) + row * a.ldy, a.cols, first, t, x);
        if (t == 0 && rank == 0) {
            if (a.mean) a.mean[row] = left == left ? mean + left : mean;   // an infinity stays
            if (a.rstd) a.rstd[row] = r;
        }
    }
}

template <class C>
cudaError_t launch_as(const NormProblem& p, cudaStream_t st) {
    const int ctas = norm_ctas<C>(p.cols);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t want = (p.rows + C::ROWS - 1) / C::ROWS, room = int64_t(sms) * (1024 / C::THREADS) / ctas;
    const ForwardArgs a{p.x, p.ldx, p.weight, p.bias, p.y, p.ldy, p.mean, p.rstd, p.rows, int32_t(p.cols), ctas, p.eps};
    return norm_launch(k_norm_forward<C>, int(want < room ? want : room), ctas, C::THREADS, 0, st, a);
}

}  // namespace

cudaError_t launch_norm_forward(const NormProblem& p, cudaStream_t st) {
    auto go = [&](auto c) { return launch_as<decltype(c)>(p, st); };
    if (p.bf16) return p.vec ? norm_dispatch<uint16_t, true>(p.cols, go) : norm_dispatch<uint16_t, false>(p.cols, go);
    return p.vec ? norm_dispatch<float, true>(p.cols, go) : norm_dispatch<float, false>(p.cols, go);
}

}  // namespace fsdp
