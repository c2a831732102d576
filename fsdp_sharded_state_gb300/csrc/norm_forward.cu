// norm_forward.cu -- y = (x - mean) * rstd * weight + bias, row by row.
//
// Bound by HBM: x read and y written once.  A row stays in registers; its mean is summed first
// and the squares of what is left after it, so that a common offset of the row costs no digits.
// What rounding did to the mean of an fp32 row is taken out again: with d = x - mean, the sum of d is 0 but
// for it, and where d's own mean exceeds 2^-23 of d's root mean square, as in rows far from
// zero, the variance and y are formed from d less its mean.  Elements of bf16 rows are 2^-8 of
// the offset apart or equal: the mean's 2^-24 of it is nothing beside that, or beside y's rounding.
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

// CTAs of an SM: 768 threads of up to 80 registers, or two CTAs of 512 of 64 (four of 256 threads
// spill what they hold of weight and bias).
template <class C>
constexpr int kForwardCtas = C::THREADS == 256 ? 3 : 2;

template <class C>
__global__ void __launch_bounds__(C::THREADS, kForwardCtas<C>)
k_norm_forward(const __grid_constant__ ForwardArgs a) {
    using T = typename C::T;
    using Sum = RowSum<C, 1>;
    using Sums = RowSum<C, 2>;                   // fp32
    extern __shared__ __align__(128) unsigned char smem_raw[];   // the rings
    __shared__ __align__(16) float sums[C::GW > 1 ? (Sum::FLOATS + Sums::FLOATS) * C::SIDE : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid % C::G;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    RowRing<C, 1> ring = make_ring<C, 1>(smem_raw, warp, first, a.cols, a.stages, a.block, a.wait_ns);
    ring.base[0] = static_cast<const T*>(a.x) + first;
    ring.ld[0] = a.ldx;
    const bool issuer = C::GW == 1 || t == 0;
    if (C::GW == 1 ? lane == 0 : t == 0) ring.init();
    if constexpr (C::CLUSTER) {                  // no CTA writes to another that has not started
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    pdl_wait();
    // blocks of rows go to the groups in turn
    const int64_t step = int64_t(gridDim.x / a.ctas) * C::SIDE * a.block;
    const int64_t row0 = (int64_t(blockIdx.x / a.ctas) * C::SIDE + warp / C::GW) * a.block;
    if (issuer) {
        for (int s = 0; s < a.stages; ++s)
            if (row0 + s * step < a.rows) ring.fetch(row0 + s * step, a.rows, s, lane);
    }
    pair w[C::P], b[C::P];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
    norm_vector<C>(static_cast<const T*>(a.bias), a.cols, first, t, 0.f, b);
    Sum sum{sums};
    Sums sum2{sums + (C::GW > 1 ? Sum::FLOATS * C::SIDE : 0)};
    const bool full = norm_full<C>(a.cols, first, t);
    const float n = float(a.cols), over_n = 1.f / n;
    int s = 0;
    uint32_t phase = 0;
    auto next_stage = [&](int64_t row) {
        if (issuer && row + a.stages * step < a.rows) ring.fetch(row + a.stages * step, a.rows, s, lane);
        if (++s == a.stages) {
            s = 0;
            phase ^= 1;
        }
    };
    // the threads of a group, or of a cluster, leave the loops together
    for (int64_t row = row0; row < a.rows; row += step) {
        ring.wait(s, phase);
        const int count = a.rows - row < a.block ? int(a.rows - row) : a.block;
        for (int j0 = 0; j0 < count; j0 += C::GW == 1 ? 32 / C::L : 1) {
            const int j = j0 + (C::GW == 1 ? lane / C::L : 0);
            const bool have = j < count;
            pair x[C::P];
            if (have) {
                norm_load<C>(ring.row_of(row + j, j, s, 0), a.cols, first, t, full, x);
            } else {
#pragma unroll
                for (int i = 0; i < C::P; ++i) x[i] = 0;
            }
            pair p = x[0];
#pragma unroll
            for (int i = 1; i < C::P; ++i) p = add2(p, x[i]);
            float v[1] = {both(p)};
            sum(v, warp, lane, a.ctas);
            if (C::GW > 1) next_stage(row);      // every thread has read the stage
            const float mean = v[0] / n;         // exact in rows of one value
            const pair minus = pair_of(-mean, -mean);
#pragma unroll
            for (int i = 0; i < C::P; ++i) x[i] = add2(x[i], minus);
            if (!full) norm_trim<C>(a.cols, first, t, x);
            pair q = mul2(x[0], x[0]);
#pragma unroll
            for (int i = 1; i < C::P; ++i) q = fma2(x[i], x[i], q);
            float var, left = 0.f;
            if constexpr (sizeof(T) == 2) {
                v[0] = both(q);
                sum(v, warp, lane, a.ctas);
                var = v[0] * over_n;
            } else {
                p = x[0];
#pragma unroll
                for (int i = 1; i < C::P; ++i) p = add2(p, x[i]);
                float d[2] = {both(p), both(q)};
                sum2(d, warp, lane, a.ctas);
                // what the sum left of an offset far beyond the spread; below that it is the roundings
                // of the differences themselves, which need not average out
                left = d[0] * over_n;
                if (left * left <= 1.5e-14f * (d[1] * over_n)) left = 0.f;
                var = (d[1] - d[0] * left) * over_n;
                if (var < 0.f) var = 0.f;        // a NaN stays
            }
            const float rstd = __frsqrt_rn(var + a.eps);
            if (!have) continue;
            if (sizeof(T) == 4 && left != 0.f) {
                const pair l = pair_of(-left, -left);
#pragma unroll
                for (int i = 0; i < C::P; ++i) x[i] = add2(x[i], l);
            }
            const pair r = pair_of(rstd, rstd);
#pragma unroll
            for (int i = 0; i < C::P; ++i) x[i] = fma2(mul2(x[i], r), w[i], b[i]);
            norm_store<C>(static_cast<T*>(a.y) + (row + j) * a.ldy, a.cols, first, t, full, x);
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
    const int ctas = norm_ctas<C>(p.cols), per_sm = kForwardCtas<C>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = norm_prepare(k_norm_forward<C>, prepared, dev);
    if (e != cudaSuccess) return e;
    const RingShape ring = ring_shape<C>(1, p.cols, per_sm);
    const int64_t each = ring.block * C::SIDE;
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
