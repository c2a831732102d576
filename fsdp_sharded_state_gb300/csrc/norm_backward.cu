// norm_backward.cu -- the gradients of a layer norm.
//
// With h = (x - mean) * rstd and g = dy * weight:
//     dx = residual + rstd * (g - mean over the row of g - h * mean over the row of g h)
//     dw (+)= sum over rows of dy h;   db (+)= sum over rows of dy
//
// Bound by HBM: x, dy and the residual read, dx written once.  dw and db cost no second pass: a
// thread keeps its columns of every row that its CTA works on, adds them up in fp32 registers,
// and leaves one row of partial sums per CTA, which k_norm_join adds up in a fixed order.
#include "norm_rows.cuh"

namespace fsdp {
namespace {

struct BackwardArgs {
    const void* x;
    int64_t ldx;
    const void* dy;
    int64_t lddy;
    const void* weight;
    const void* residual;
    int64_t ldr;
    const float* mean;
    const float* rstd;
    void* dx;
    int64_t lddx;
    float* partial;                 // [2][groups][pitch], or NULL
    int64_t pitch, rows;
    int32_t cols, ctas, stages, block;
    uint64_t wait_ns;
};

// Columns of a row of partial sums.
__host__ __device__ inline int64_t partial_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

template <class C>
__global__ void __launch_bounds__(C::THREADS, 512 / C::THREADS)
k_norm_backward(const __grid_constant__ BackwardArgs a) {
    using T = typename C::T;
    using Sums = RowSum<C, 2>;
    extern __shared__ __align__(128) unsigned char smem_raw[];   // the rings; at the end a row of sums per group
    __shared__ __align__(16) float sums[C::GW > 1 ? Sums::FLOATS * C::SIDE : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid % C::G;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    const int part = blockIdx.x / a.ctas, parts = gridDim.x / a.ctas;
    const bool res = a.residual != nullptr;
    RowRing<C, 3> ring = make_ring<C, 3>(smem_raw, warp, first, a.cols, a.stages, a.block, a.wait_ns);
    ring.base[0] = static_cast<const T*>(a.x) + first;
    ring.base[1] = static_cast<const T*>(a.dy) + first;
    ring.base[2] = res ? static_cast<const T*>(a.residual) + first : nullptr;
    ring.ld[0] = a.ldx;
    ring.ld[1] = a.lddy;
    ring.ld[2] = a.ldr;
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
    const int64_t step = int64_t(parts) * C::SIDE * a.block;
    const int64_t row0 = (int64_t(part) * C::SIDE + warp / C::GW) * a.block;
    if (issuer) {
        for (int s = 0; s < a.stages; ++s)
            if (row0 + s * step < a.rows) ring.fetch(row0 + s * step, a.rows, s, lane);
    }
    pair w[C::P], dw[C::P], db[C::P];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
#pragma unroll
    for (int i = 0; i < C::P; ++i) dw[i] = db[i] = 0;
    Sums sum{sums};
    const bool full = norm_full<C>(a.cols, first, t);
    const float over_n = 1.f / float(a.cols);
    int s = 0;
    uint32_t phase = 0;
    auto next_stage = [&](int64_t row) {
        if (issuer && row + a.stages * step < a.rows) ring.fetch(row + a.stages * step, a.rows, s, lane);
        if (++s == a.stages) {
            s = 0;
            phase ^= 1;
        }
    };
    // mean and rstd are read a block ahead: of its row lane by lane l, where a block is a warp's
    float next_mean = 0.f, next_rstd = 0.f;
    auto read_ahead = [&](int64_t row) {
        if (C::GW == 1 ? lane < a.block && row + lane < a.rows : row < a.rows) {
            next_mean = a.mean[row + (C::GW == 1 ? lane : 0)];
            next_rstd = a.rstd[row + (C::GW == 1 ? lane : 0)];
        }
    };
    read_ahead(row0);
    // the threads of a group, or of a cluster, leave the loops together
    for (int64_t row = row0; row < a.rows; row += step) {
        const float row_mean = next_mean, row_rstd = next_rstd;
        read_ahead(row + step);
        const int count = a.rows - row < a.block ? int(a.rows - row) : a.block;
        if (C::GW == 1) ring.wait(s, phase);
        for (int j0 = 0; j0 < count; j0 += C::GW == 1 ? 32 / C::L : 1) {
            const int j = j0 + (C::GW == 1 ? lane / C::L : 0);
            const bool have = j < count;
            pair h[C::P], g[C::P], add[C::P];
            float v[2] = {0.f, 0.f}, mean = row_mean, rstd = row_rstd;
            if constexpr (C::GW == 1) {
                mean = __shfl_sync(0xffffffffu, row_mean, j & 31);
                rstd = __shfl_sync(0xffffffffu, row_rstd, j & 31);
            }
            if (have) {
                if (C::GW > 1) ring.wait(s, phase);
                norm_load<C>(ring.row_of(row + j, j, s, 0), a.cols, first, t, full, h);
                norm_load<C>(ring.row_of(row + j, j, s, 1), a.cols, first, t, full, g);
                if (res) norm_load<C>(ring.row_of(row + j, j, s, 2), a.cols, first, t, full, add);
                const pair m = pair_of(-mean, -mean), r = pair_of(rstd, rstd);
#pragma unroll
                for (int i = 0; i < C::P; ++i) h[i] = mul2(add2(h[i], m), r);
                if (!full) norm_trim<C>(a.cols, first, t, h);
                pair p = 0, q = 0;
#pragma unroll
                for (int i = 0; i < C::P; ++i) {
                    dw[i] = fma2(g[i], h[i], dw[i]);
                    db[i] = add2(db[i], g[i]);
                    g[i] = mul2(g[i], w[i]);
                    p = add2(p, g[i]);
                    q = fma2(g[i], h[i], q);
                }
                v[0] = both(p);
                v[1] = both(q);
            }
            sum(v, warp, lane, a.ctas);
            if (C::GW > 1) next_stage(row);      // every thread has read the stage
            if (!have) continue;
            const float c0 = -v[0] * over_n, c1 = -v[1] * over_n;
            const pair m0 = pair_of(c0, c0), m1 = pair_of(c1, c1), r = pair_of(rstd, rstd);
            if (res) {
#pragma unroll
                for (int i = 0; i < C::P; ++i) g[i] = fma2(fma2(h[i], m1, add2(g[i], m0)), r, add[i]);
            } else {
#pragma unroll
                for (int i = 0; i < C::P; ++i) g[i] = mul2(fma2(h[i], m1, add2(g[i], m0)), r);
            }
            norm_store<C>(static_cast<T*>(a.dx) + (row + j) * a.lddx, a.cols, first, t, full, g);
        }
        if (C::GW == 1) {
            __syncwarp();                        // every lane has read the stage
            next_stage(row);
        }
    }
    ring.leave();
    if (!a.partial) return;
    float* const out_w = a.partial + part * a.pitch;
    float* const out_b = out_w + parts * a.pitch;
    if constexpr (C::SIDE > 1) {
        // the rows of a warp, then the groups of the CTA, in order
        float* const smem = reinterpret_cast<float*>(smem_raw);
#pragma unroll
        for (int o = 16; o >= C::L; o >>= 1)
#pragma unroll
            for (int i = 0; i < C::P; ++i) {
                dw[i] = add2(dw[i], __shfl_xor_sync(0xffffffffu, dw[i], o));
                db[i] = add2(db[i], __shfl_xor_sync(0xffffffffu, db[i], o));
            }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            if (C::GW > 1 || lane < C::L) {
#pragma unroll
                for (int e = 0; e < C::E; e += 2) {
                    const float2 f = split(which ? db[e / 2] : dw[e / 2]);
                    smem[warp / C::GW * C::COLS + norm_col<C>(0, t, e)] = f.x;
                    smem[warp / C::GW * C::COLS + norm_col<C>(0, t, e + 1)] = f.y;
                }
            }
            __syncthreads();
            for (int c = tid; c < a.cols; c += C::THREADS) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < C::SIDE; ++k) v += smem[k * C::COLS + c];
                (which ? out_b : out_w)[c] = v;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int c = norm_col<C>(first, t, e);
            if (c < a.cols) {
                const float2 f = split(dw[e / 2]), g = split(db[e / 2]);
                out_w[c] = e & 1 ? f.y : f.x;
                out_b[c] = e & 1 ? g.y : g.x;
            }
        }
    }
}

// out[c] (+)= the sum over p of part[p][c], for dw and (blockIdx.y = 1) db.  A block takes 32
// columns; its kJoinWarps warps every kJoinWarps-th row each, and then warp 0 adds the warps'
// sums up in order.
constexpr int kJoinWarps = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps)
k_norm_join(const float* part, int parts, int64_t pitch, int cols, T* dw, T* db, bool accumulate) {
    __shared__ float sums[kJoinWarps][32];
    pdl_wait();
    T* const out = blockIdx.y ? db : dw;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* const src = part + (blockIdx.y ? parts * pitch : 0);
    float v = 0.f;
    if (out && c < cols) {
#pragma unroll 10
        for (int p = warp; p < parts; p += kJoinWarps) v += src[p * pitch + c];
    }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && out && c < cols) {
        v = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) v += sums[k][lane];
        if (accumulate) v += norm_get(out + c);
        norm_put(out + c, v);
    }
}

// CTAs (or clusters) that work through the rows, each with a row of partial sums: as many as
// fit the 152 SMs at once, fewer where there are few rows.
template <class C>
int64_t backward_groups(int64_t rows, int64_t cols) {
    const int64_t each = ring_shape<C>(3, cols, 512 / C::THREADS).block * C::SIDE;
    const int64_t want = (rows + each - 1) / each, room = 152 * (512 / C::THREADS) / norm_ctas<C>(cols);
    return want < room ? want : room;
}

template <class C>
cudaError_t launch_as(const NormProblem& p, cudaStream_t st) {
    const int ctas = norm_ctas<C>(p.cols);
    const int64_t groups = backward_groups<C>(p.rows, p.cols), pitch = partial_pitch(p.cols);
    const bool sums = p.dw || p.db;
    cudaError_t e = cudaSuccess;
    if (p.rows > 0) {
        static std::atomic<uint64_t> prepared{0};
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess || (e = norm_prepare(k_norm_backward<C>, prepared, dev)) != cudaSuccess) return e;
        const RingShape ring = ring_shape<C>(3, p.cols, 512 / C::THREADS);
        const size_t last = C::SIDE > 1 ? size_t(C::SIDE) * C::COLS * 4 : 0;
        const BackwardArgs a{p.x, p.ldx, p.dy, p.lddy, p.weight, p.residual, p.ldr, p.mean, p.rstd, p.y, p.ldy,
                             sums ? p.partial : nullptr, pitch, p.rows, int32_t(p.cols), ctas, ring.stages, ring.block, detail::kWaitNs};
        e = norm_launch(k_norm_backward<C>, int(groups), ctas, C::THREADS, ring.bytes > last ? ring.bytes : last, st, a);
    }
    if (e != cudaSuccess || !sums || (p.rows == 0 && p.accumulate)) return e;
    const dim3 grid(unsigned((p.cols + 31) / 32), 2);
    if (p.grad_bf16)
        return launch(k_norm_join<uint16_t>, grid, dim3(32 * kJoinWarps), 0, st, static_cast<const float*>(p.partial), int(groups), pitch,
                      int(p.cols), static_cast<uint16_t*>(p.dw), static_cast<uint16_t*>(p.db), p.accumulate);
    return launch(k_norm_join<float>, grid, dim3(32 * kJoinWarps), 0, st, static_cast<const float*>(p.partial), int(groups), pitch,
                  int(p.cols), static_cast<float*>(p.dw), static_cast<float*>(p.db), p.accumulate);
}

}  // namespace

int64_t norm_partial_floats(int64_t rows, int64_t cols) {
    int64_t groups = 0;
    auto most = [&](auto c) {
        const int64_t g = backward_groups<decltype(c)>(rows, cols);
        if (g > groups) groups = g;
        return cudaSuccess;
    };
    norm_dispatch<float, true>(cols, most);
    norm_dispatch<uint16_t, true>(cols, most);
    return 2 * groups * partial_pitch(cols);
}

cudaError_t take_wait_error_norm_backward(unsigned int* flag) { return take_norm_wait_error(flag); }

cudaError_t launch_norm_backward(const NormProblem& p, cudaStream_t st) {
    auto go = [&](auto c) { return launch_as<decltype(c)>(p, st); };
    if (p.bf16) return p.vec ? norm_dispatch<uint16_t, true>(p.cols, go) : norm_dispatch<uint16_t, false>(p.cols, go);
    return p.vec ? norm_dispatch<float, true>(p.cols, go) : norm_dispatch<float, false>(p.cols, go);
}

}  // namespace fsdp
