// linear_skinny.cu -- forward and dgrad of a few rows (a single token, a short prompt): the
// weight is read once, in fp32 FMAs, where the tensor cores' tiles would be empty and fp32
// weights would have to be split first.
//
// Bound by the weight's bytes.  Products and sums are fp32; the order of a sum depends on the
// sizes alone.
#include "linear_launch.cuh"

namespace fsdp {
namespace {

constexpr int kSkThreads = 256, kSkWarps = kSkThreads / 32;

// Elements a lane takes of a row at a time: 16 bytes; in one access where the row is aligned
// (lane l: E l ..), else strided over the warp (l, 32 + l, ..).
template <typename T, bool VEC>
struct Lane {
    static constexpr int E = 16 / sizeof(T);
    static __device__ __forceinline__ void load(const T* row, int64_t k0, int64_t K, int lane, float (&v)[E]) {
        if constexpr (VEC) {
            const int64_t k = k0 + lane * E;
            if (k + E <= K) {
                if constexpr (E == 8) {
                    widen(load_raw(reinterpret_cast<const uint16_t*>(row + k)), v);
                } else {
                    const float4 q = ld4(reinterpret_cast<const float*>(row + k));
                    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                }
                return;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = k + e < K ? load1(row + k + e) : 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = k0 + lane + 32 * e < K ? load1(row + k0 + lane + 32 * e) : 0.f;
        }
    }
};

// The epilogue of one element.
template <int MODE, typename T>
__device__ __forceinline__ void emit_one(const LinEpi& ep, int64_t row, int64_t col, float x) {
    float v[1] = {x};
    if constexpr (MODE == kForward) {
        if (ep.bias) v[0] += load1(static_cast<const T*>(ep.bias) + col);
        if (ep.preact) store1(static_cast<T*>(ep.preact) + row * ep.ldz + col, v[0]);
        activate<false, 1>(v, ep.act);
    }
    if (ep.drop.on) {
        const uint4 w = drop_words(ep.drop, row, col >> 2);
        const int k = int(col & 3);
        v[0] = drop1(ep.drop, k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w, v[0]);
    }
    if constexpr (MODE == kDgrad) {
        if (ep.act != FSDP_ACT_NONE) {
            const float z[1] = {load1(static_cast<const T*>(ep.preact) + row * ep.ldz + col)};
            activate_grad<false, 1>(v, z, ep.act);
        }
    }
    if (ep.residual) v[0] += load1(static_cast<const T*>(ep.residual) + row * ep.ldr + col);
    store1(static_cast<T*>(ep.out) + row * ep.ldo + col, v[0]);
}

// The sum over the warp's lanes of N values each: afterwards lane l holds the sums of the
// values sum_index(l) .. in v[0 .. max(N / 32, 1)).  Halving exchanges: N - N / 32 shuffles.
template <int N>
__device__ __forceinline__ void lane_sums(float (&v)[N], int lane) {
    int n = N;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) {
        if (n > 1) {
            n >>= 1;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < n) {
                    const float keep = lane & s ? v[i + n] : v[i], send = lane & s ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
        }
    }
}
// The index of the first value that lane l holds afterwards.
template <int N>
__device__ __forceinline__ int sum_index(int lane) {
    int n = N, at = 0;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) {
        if (n > 1) {
            n >>= 1;
            at += lane & s ? n : 0;
        }
    }
    return at;
}

// forward: a CTA takes F out-features of TB rows; its 8 warps share K in steps of 32 lanes of
// 16 bytes, then join through shared memory.
template <typename T, int TB, int F, bool VEC>
__global__ void __launch_bounds__(kSkThreads)
k_skinny_forward(const T* __restrict__ x, int64_t ldx, const T* __restrict__ w, int64_t ldw, int64_t K,
                 const __grid_constant__ LinEpi ep) {
    constexpr int E = Lane<T, VEC>::E, N = TB * F;
    __shared__ float part[kSkWarps][N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t f0 = int64_t(blockIdx.x) * F, t0 = int64_t(blockIdx.y) * TB;
    pdl_wait();
    float acc[N] = {};
#pragma unroll 1
    for (int64_t k0 = int64_t(warp) * 32 * E; k0 < K; k0 += kSkWarps * 32 * E) {
        float wv[F][E], xv[E];
#pragma unroll
        for (int f = 0; f < F; ++f) {            // past the last feature: its row again, not kept
            const int64_t r = f0 + f < ep.cols ? f0 + f : ep.cols - 1;
            Lane<T, VEC>::load(w + r * ldw, k0, K, lane, wv[f]);
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const int64_t r = t0 + t < ep.rows ? t0 + t : ep.rows - 1;
            Lane<T, VEC>::load(x + r * ldx, k0, K, lane, xv);
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[t * F + f] = __fmaf_rn(xv[e], wv[f][e], acc[t * F + f]);
        }
    }
    lane_sums<N>(acc, lane);
    constexpr int HELD = N / 32 > 1 ? N / 32 : 1;
    const int at = sum_index<N>(lane);
#pragma unroll
    for (int i = 0; i < HELD; ++i) part[warp][at + i] = acc[i];    // with N < 32, several lanes write the same sum
    __syncthreads();
    if (threadIdx.x < N) {
        float t = part[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < kSkWarps; ++k) t += part[k][threadIdx.x];
        const int64_t row = t0 + threadIdx.x / F, col = f0 + threadIdx.x % F;
        if (row < ep.rows && col < ep.cols) emit_one<kForward, T>(ep, row, col, t);
    }
}

// dgrad: a cluster of 8 CTAs takes 32 E in-features of TB rows; its 64 warps share the
// out-features (the rows of w), a lane holding E columns; the CTAs' sums join in the CTA that
// owns an eighth of the columns.  A CTA's shared memory may be written once the CTA has started:
// each arrives at the cluster's barrier first and waits there after its share of the weight.
constexpr int kSkRanks = 8;
template <typename T, int TB, bool VEC>
__global__ void __launch_bounds__(kSkThreads)
k_skinny_dgrad(const T* __restrict__ dz, int64_t lddz, const T* __restrict__ w, int64_t ldw, int64_t K,
               const __grid_constant__ LinEpi ep) {
    constexpr int E = Lane<T, VEC>::E, COLS = 32 * E, OWN = COLS / kSkRanks, U = TB <= 2 ? 8 : 4;
    __shared__ float warps[kSkWarps][COLS];
    __shared__ float ranks[kSkRanks][TB][OWN];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t c0 = int64_t(blockIdx.x / kSkRanks) * COLS, t0 = int64_t(blockIdx.y) * TB;
    cluster_arrive();
    pdl_wait();
    float acc[TB][E] = {};
    constexpr int64_t STEP = kSkWarps * kSkRanks;
#pragma unroll 1
    for (int64_t o = int64_t(rank) * kSkWarps + warp; o < K; o += U * STEP) {
        float wv[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = o + u * STEP < K ? o + u * STEP : K - 1;
            Lane<T, VEC>::load(w + r * ldw + c0, 0, ep.cols - c0, lane, wv[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int64_t row = t0 + t < ep.rows ? t0 + t : ep.rows - 1;
                const float g = o + u * STEP < K ? load1(dz + row * lddz + o + u * STEP) : 0.f;
                // the last row again, past the end: kept out by a select, not by a product with 0
#pragma unroll
                for (int e = 0; e < E; ++e) acc[t][e] = __fmaf_rn(g, o + u * STEP < K ? wv[u][e] : 0.f, acc[t][e]);
            }
        }
    }
    __syncwarp();
    cluster_wait();
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) warps[warp][VEC ? lane * E + e : lane + 32 * e] = acc[t][e];
        __syncthreads();
        if (threadIdx.x < COLS) {
            float s = warps[0][threadIdx.x];
#pragma unroll
            for (int k = 1; k < kSkWarps; ++k) s += warps[k][threadIdx.x];
            st_cluster(map_rank(smem_addr(&ranks[rank][t][threadIdx.x % OWN]), threadIdx.x / OWN), s);
        }
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (threadIdx.x < TB * OWN) {
        const int t = threadIdx.x / OWN, c = threadIdx.x % OWN;
        float s = ranks[0][t][c];
#pragma unroll
        for (int k = 1; k < kSkRanks; ++k) s += ranks[k][t][c];
        const int64_t row = t0 + t, col = c0 + rank * OWN + c;
        if (row < ep.rows && col < ep.cols) emit_one<kDgrad, T>(ep, row, col, s);
    }
}

template <typename T, int TB, int F, bool VEC>
cudaError_t forward_as(const SkinnyProblem& p, cudaStream_t st) {
    const int64_t bx = ceil_div(p.epi.cols, F), by = ceil_div(p.epi.rows, TB);
    if (bx > INT32_MAX || by > 65535) return cudaErrorInvalidValue;
    return launch(k_skinny_forward<T, TB, F, VEC>, dim3(unsigned(bx), unsigned(by)), dim3(kSkThreads), 0, st,
                  static_cast<const T*>(p.x), p.ldx, static_cast<const T*>(p.w), p.ldw, p.K, p.epi);
}
template <typename T, int TB, bool VEC>
cudaError_t dgrad_as(const SkinnyProblem& p, cudaStream_t st) {
    const int64_t bx = ceil_div(p.epi.cols, 32 * Lane<T, VEC>::E) * kSkRanks, by = ceil_div(p.epi.rows, TB);
    if (bx > INT32_MAX || by > 65535) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSkRanks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(bx), unsigned(by));
    cfg.blockDim = dim3(kSkThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_skinny_dgrad<T, TB, VEC>, static_cast<const T*>(p.x), p.ldx, static_cast<const T*>(p.w), p.ldw,
                              p.K, p.epi);
}

template <typename T, bool VEC>
cudaError_t forward_rows(const SkinnyProblem& p, cudaStream_t st) {
    const int64_t rows = p.epi.rows;
    if (rows == 1) return forward_as<T, 1, 8, VEC>(p, st);
    if (rows == 2) return forward_as<T, 2, 8, VEC>(p, st);
    return forward_as<T, 4, 8, VEC>(p, st);       // more than 4: the weight again, from L2
}
template <bool VEC>
cudaError_t dgrad_rows(const SkinnyProblem& p, cudaStream_t st) {
    return p.epi.rows == 1   ? dgrad_as<float, 1, VEC>(p, st)
           : p.epi.rows == 2 ? dgrad_as<float, 2, VEC>(p, st)
                             : dgrad_as<float, 4, VEC>(p, st);
}

}  // namespace

cudaError_t launch_skinny(const SkinnyProblem& p, cudaStream_t st) {
    auto rows16 = [&](const void* q, int64_t ld, int es) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld * es % 16 == 0; };
    const int es = p.bf16 ? 2 : 4;
    // forward reads rows of both along K, dgrad rows of w along the columns
    const bool vec = rows16(p.w, p.ldw, es) && (p.mode == kDgrad || rows16(p.x, p.ldx, es));
    if (p.mode == kDgrad) return vec ? dgrad_rows<true>(p, st) : dgrad_rows<false>(p, st);
    if (p.bf16) return vec ? forward_rows<uint16_t, true>(p, st) : forward_rows<uint16_t, false>(p, st);
    return vec ? forward_rows<float, true>(p, st) : forward_rows<float, false>(p, st);
}

// Measured on GB300 (us, this file / the tensor cores), weight 6432 x 3776 (floors 14.3 fp32,
// 7.2 bf16): forward fp32 1 row 21 / 67, 4 rows 22 / 67, 12 rows 47 / 67; dgrad fp32 1 row 25 /
// 70, 4 rows 36 / 70, 8 rows two passes of that; forward bf16 1 row 13.7 / 12.6, 4 rows 27 /
// 12.7, at 2048 x 2048 2.8 / 6.0 and 4.7 / 5.9; dgrad bf16 36 / 13.
bool use_skinny(LinMode mode, bool bf16, int64_t rows, int64_t in, int64_t out) {
    if (mode == kDgrad) return !bf16 && rows <= 4;
    if (!bf16) return rows <= 16;
    return rows <= 4 && (rows == 1 || rows * in * out <= (int64_t(1) << 24));
}

}  // namespace fsdp
