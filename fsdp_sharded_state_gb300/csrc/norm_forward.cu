// norm_forward.cu -- y = (x - mean) * rstd * weight + bias, row by row.
//
// Bound by HBM: x read and y written once.  A row stays in registers; its mean is summed first
// and the squares of what is left after it, so that a common offset of the row costs no digits.
// What rounding did to the mean is taken out again: with d = x - mean, the sum of d is 0 but for it,
// and the variance and y are formed from d less its mean.  In fp32 that is where d's own mean exceeds
// 2^-23 of d's root mean square.  In bf16 rows only a mean far beyond the spread can do it: where few
// of many equal elements deviate, by 2^-8 of the offset or more, the others differ from the mean by far less
// (5 of 11008 one step above 4992: y 0.8 % off).  Rows whose mean is above four times the root mean square of
// d take one more sum; the mean of the others is off by no more than the sum of d would be.
//
// bf16, one GB300: 16384 x 4096 46 us (0.86 of the copy rate; 52 with the sum that rows far from zero take),
// 65536 x 256 14.5 (0.68: neither HBM nor the issue of instructions, 60 %, is full), 4096 x 16384 47; fp32 8192 x 4096 48.
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

// CTAs of an SM: threads of up to 80 registers, or 128 where they hold 32 columns.
template <class C>
constexpr int kForwardCtas = C::V == 4 ? 512 / C::THREADS : 768 / C::THREADS;

template <class C>
__global__ void __launch_bounds__(C::THREADS, kForwardCtas<C>)
k_norm_forward(const __grid_constant__ ForwardArgs a) {
    using T = typename C::T;
    using Sum = RowSum<C, 1>;
    using Sums = RowSum<C, 2>;                   // fp32
    extern __shared__ __align__(128) unsigned char smem_raw[];   // the ring
    __shared__ __align__(16) float sums[C::GW > 1 ? (Sum::FLOATS + Sums::FLOATS) * C::SIDE : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid % C::G, group = warp / C::GW;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    const uint32_t rows = uint32_t(a.rows), row0 = blockIdx.x / a.ctas * uint32_t(C::SIDE * a.block);
    RowRing<C, 1> ring(smem_raw, first, a.cols, a.stages, a.block, rows, gridDim.x / a.ctas * uint32_t(C::SIDE * a.block), a.wait_ns);
    ring.matrix(0, a.x, a.ldx, first, row0);
    if (tid == 0) ring.init();
    if constexpr (C::CLUSTER) {                  // no CTA writes to another that has not started
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    pdl_wait();
    if (C::SIDE == 1 ? tid == 0 : warp == 0) ring.begin(row0, lane);
    pair w[C::P], b[C::P];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
    norm_vector<C>(static_cast<const T*>(a.bias), a.cols, first, t, 0.f, b);
    Sum sum{sums, ring.sums(0), a.wait_ns};
    Sums sum2{sums + (C::GW > 1 ? Sum::FLOATS * C::SIDE : 0), ring.sums(1), a.wait_ns};
    const bool full = __all_sync(0xffffffffu, norm_full<C>(a.cols, first, t));
    const float n = float(a.cols), over_n = 1.f / n;
    // of the group's first row of the stage: its place in it and in y
    const int j1 = group * (C::GW == 1 ? a.block : 1) + (C::GW == 1 ? lane / C::L : 0);
    const int block = C::GW == 1 ? a.block : 1;
    uint32_t mine = row0 + j1;
    T* py = static_cast<T*>(a.y) + mine * a.ldy;
    const int64_t y_step = ring.step * a.ldy, y_side = (32 / C::L) * a.ldy;
    // the threads of a CTA, or of a cluster, leave the loop together
    for (uint32_t row = row0; row < rows; row += ring.step, mine += ring.step, py += y_step) {
        ring.wait();
        T* y = py;
        for (int j0 = 0; j0 < block; j0 += C::GW == 1 ? 32 / C::L : 1, y += y_side) {
            const bool have = mine + j0 < rows;
            pair x[C::P];
            if (have) {
                norm_load<C>(ring.row_of(j1 + j0, 0), a.cols, first, t, full, x);
            } else {
#pragma unroll
                for (int i = 0; i < C::P; ++i) x[i] = 0;
            }
            pair p = x[0];
#pragma unroll
            for (int i = 1; i < C::P; ++i) p = add2(p, x[i]);
            float v[1] = {both(p)};
            sum(v, warp, lane, a.ctas);
            if (C::GW > 1) {                     // every thread of the group has read its row
                if (C::SIDE == 1 ? tid == 0 : warp % C::GW == 0) ring.release(row, lane);
                ring.next();
            }
            // the quotient by n, its rounding taken out: exact in rows of one value
            float mean = v[0] * over_n;
            if (fabsf(mean) < 1e38f) mean = __fmaf_rn(__fmaf_rn(-mean, n, v[0]), over_n, mean);
            const pair minus = pair_of(-mean, -mean);
#pragma unroll
            for (int i = 0; i < C::P; ++i) x[i] = add2(x[i], minus);
            if (!full) norm_trim<C>(a.cols, first, t, x);
            pair q = mul2(x[0], x[0]);
#pragma unroll
            for (int i = 1; i < C::P; ++i) q = fma2(x[i], x[i], q);
            float var, left = 0.f;
            auto sum_of_d = [&]() {
                pair p = x[0];
#pragma unroll
                for (int i = 1; i < C::P; ++i) p = add2(p, x[i]);
                return both(p);
            };
            if constexpr (sizeof(T) == 2) {
                v[0] = both(q);
                sum(v, warp, lane, a.ctas);
                var = v[0] * over_n;
                // the same in all threads of a row; other rows of the warp go along and subtract 0
                const bool far = mean * mean > 16.f * var;
                if (__builtin_expect(__any_sync(0xffffffffu, far), 0)) {
                    v[0] = sum_of_d();
                    sum(v, warp, lane, a.ctas);
                    const float l = far ? v[0] * over_n : 0.f;
                    const pair less = pair_of(-l, -l);
#pragma unroll
                    for (int i = 0; i < C::P; ++i) x[i] = add2(x[i], less);
                    if (far) {
                        mean += l;
                        var = fmaxf(var - l * l, 0.f);
                    }
                }
            } else {
                float d[2] = {sum_of_d(), both(q)};
                sum2(d, warp, lane, a.ctas);
                // what the sum left of an offset far beyond the spread; below that it is the roundings
                // of the differences themselves, which need not average out
                left = d[0] * over_n;
                if (left * left <= 1.5e-14f * (d[1] * over_n)) left = 0.f;
                var = (d[1] - d[0] * left) * over_n;
                if (var < 0.f) var = 0.f;        // a NaN stays
            }
            // CUDA's reciprocal square root (2 units in the last place), and a Newton step
            const float e = var + a.eps;
            float rstd = rsqrtf(e);
            if (rstd < 1e18f && rstd > 0.f) rstd = __fmaf_rn(0.5f * rstd, __fmaf_rn(-e * rstd, rstd, 1.f), rstd);
            if (!have) continue;
            if (sizeof(T) == 4 && left != 0.f) {
                const pair l = pair_of(-left, -left);
#pragma unroll
                for (int i = 0; i < C::P; ++i) x[i] = add2(x[i], l);
            }
            const pair r = pair_of(rstd, rstd);
#pragma unroll
            for (int i = 0; i < C::P; ++i) x[i] = fma2(mul2(x[i], r), w[i], b[i]);
            norm_store<C>(y, a.cols, first, t, full, x);
            if (t == 0 && rank == 0) {
                if (a.mean) a.mean[mine + j0] = left == left ? mean + left : mean;   // an infinity stays
                if (a.rstd) a.rstd[mine + j0] = rstd;
            }
        }
        if (C::GW == 1) {
            __syncwarp();                        // every lane has read the warp's rows
            ring.release(row, lane);
            ring.next();
        }
    }
    ring.leave(C::CLUSTER ? sum.wait_ns && sum2.wait_ns : 1);
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
    if (p.bf16) return p.vec ? norm_dispatch_forward<uint16_t, true>(p.cols, go) : norm_dispatch_forward<uint16_t, false>(p.cols, go);
    return p.vec ? norm_dispatch_forward<float, true>(p.cols, go) : norm_dispatch_forward<float, false>(p.cols, go);
}

cudaError_t take_wait_error_norm_forward(unsigned int* flag) { return take_norm_wait_error(flag); }

}  // namespace fsdp
