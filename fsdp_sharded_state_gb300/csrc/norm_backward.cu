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
    int32_t cols, ctas;
};

// Columns of a row of partial sums.
__host__ __device__ inline int64_t partial_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

template <class C>
constexpr int backward_smem() {
    return C::GW == 1 ? 8 * C::COLS * 4 : 4 * kNormMaxWarps * 4;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS)
k_norm_backward(const __grid_constant__ BackwardArgs a) {
    using T = typename C::T;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float* const smem = reinterpret_cast<float*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    const int group = blockIdx.x / a.ctas, groups = gridDim.x / a.ctas;
    if constexpr (C::CLUSTER) {                  // no CTA writes to another that has not started
        cluster_arrive();
        cluster_wait();
    }
    pdl_wait();
    float w[C::E], dw[C::E], db[C::E];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
#pragma unroll
    for (int e = 0; e < C::E; ++e) dw[e] = db[e] = 0.f;
    RowSum<C, 2> sum{smem};
    const float n = float(a.cols);
    const int64_t step = int64_t(groups) * C::ROWS;
    int64_t row = int64_t(group) * C::ROWS + (C::GW == 1 ? tid / C::L : 0);
    // the threads of a warp, CTA or cluster leave the loop together
    for (int64_t at = int64_t(group) * C::ROWS; at < a.rows; at += step, row += step) {
        const bool have = row < a.rows;
        float h[C::E], g[C::E];
        float s[2] = {0.f, 0.f}, r = 0.f;
        if (have) {
            const float mean = a.mean[row];
            r = a.rstd[row];
            norm_load<C>(static_cast<const T*>(a.x) + row * a.ldx, a.cols, first, t, h);
            norm_load<C>(static_cast<const T*>(a.dy) + row * a.lddy, a.cols, first, t, g);
#pragma unroll
            for (int e = 0; e < C::E; ++e) {
                h[e] = norm_col<C>(first, t, e) < a.cols ? (h[e] - mean) * r : 0.f;
                dw[e] = __fmaf_rn(g[e], h[e], dw[e]);
                db[e] += g[e];
                g[e] *= w[e];
                s[0] += g[e];
                s[1] = __fmaf_rn(g[e], h[e], s[1]);
            }
        }
        sum(s, warp, lane, a.ctas);
        if (!have) continue;
        const float c0 = s[0] / n, c1 = s[1] / n;
#pragma unroll
        for (int e = 0; e < C::E; ++e) g[e] = r * (g[e] - c0 - h[e] * c1);
        if (a.residual) {
            norm_load<C>(static_cast<const T*>(a.residual) + row * a.ldr, a.cols, first, t, h);
#pragma unroll
            for (int e = 0; e < C::E; ++e) g[e] += h[e];
        }
        norm_store<C>(static_cast<T*>(a.dx) + row * a.lddx, a.cols, first, t, g);
    }
    if (!a.partial) return;
    float* const out_w = a.partial + group * a.pitch;
    float* const out_b = out_w + groups * a.pitch;
    if constexpr (C::GW == 1) {
        // the rows of a warp, then the warps of the CTA, in order
#pragma unroll
        for (int o = 16; o >= C::L; o >>= 1)
#pragma unroll
            for (int e = 0; e < C::E; ++e) {
                dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
                db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
            }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            if (lane < C::L) {
#pragma unroll
                for (int e = 0; e < C::E; ++e) smem[warp * C::COLS + norm_col<C>(0, t, e)] = which ? db[e] : dw[e];
            }
            __syncthreads();
            for (int c = tid; c < a.cols; c += C::THREADS) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) v += smem[k * C::COLS + c];
                (which ? out_b : out_w)[c] = v;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int c = norm_col<C>(first, t, e);
            if (c < a.cols) {
                out_w[c] = dw[e];
                out_b[c] = db[e];
            }
        }
    }
}

// out[c] (+)= the sum over p of part[p][c], for dw and (blockIdx.y = 1) db.  A block takes 32
// columns; its kJoinWarps warps every kJoinWarps-th row each, and then warp 0 adds the warps'
// sums up in order.
constexpr int kJoinWarps = 16;

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
#pragma unroll 8
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

// Groups of threads that work through the rows, each with a row of partial sums: as many as
// fit the 152 SMs at once, fewer where there are few rows.
template <class C>
int64_t backward_groups(int64_t rows, int64_t cols) {
    const int64_t want = (rows + C::ROWS - 1) / C::ROWS, room = 152 * (512 / C::THREADS) / norm_ctas<C>(cols);
    return want < room ? want : room;
}

template <class C>
cudaError_t launch_as(const NormProblem& p, cudaStream_t st) {
    const int ctas = norm_ctas<C>(p.cols);
    const int64_t groups = backward_groups<C>(p.rows, p.cols), pitch = partial_pitch(p.cols);
    const bool sums = p.dw || p.db;
    cudaError_t e = cudaSuccess;
    if (p.rows > 0) {
        const BackwardArgs a{p.x, p.ldx, p.dy, p.lddy, p.weight, p.residual, p.ldr, p.mean, p.rstd, p.y, p.ldy,
                             sums ? p.partial : nullptr, pitch, p.rows, int32_t(p.cols), ctas};
        e = norm_launch(k_norm_backward<C>, int(groups), ctas, C::THREADS, backward_smem<C>(), st, a);
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
    norm_dispatch<float, true>(cols, [&](auto c) {
        groups = backward_groups<decltype(c)>(rows, cols);
        return cudaSuccess;
    });
    return 2 * groups * partial_pitch(cols);
}

cudaError_t launch_norm_backward(const NormProblem& p, cudaStream_t st) {
    auto go = [&](auto c) { return launch_as<decltype(c)>(p, st); };
    if (p.bf16) return p.vec ? norm_dispatch<uint16_t, true>(p.cols, go) : norm_dispatch<uint16_t, false>(p.cols, go);
    return p.vec ? norm_dispatch<float, true>(p.cols, go) : norm_dispatch<float, false>(p.cols, go);
}

}  // namespace fsdp
