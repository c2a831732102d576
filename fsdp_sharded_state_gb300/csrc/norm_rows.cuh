// norm_rows.cuh -- what the layer-norm kernels share: how a row is spread over threads, its
// loads and stores, and sums over it.
//
// A row belongs to a group of threads that hold it in registers from its load to its store:
// L lanes of a warp (up to 1024 columns; a warp then works on 32 / L rows), GW warps of a CTA
// (up to 8192), or GW warps in each CTA of a cluster (up to 65536).  A thread holds 8 V columns: V
// chunks of 8 neighbours where rows are aligned to 16 bytes (VEC), else 8 V single columns that
// are a group's width apart, so that a warp's loads are contiguous either way.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "norm.hpp"
#include "tc5.cuh"

namespace fsdp {
namespace {

template <typename T_, int L_, int GW_, int V_, bool VEC_, bool CLUSTER_ = false>
struct NormCfg {
    using T = T_;
    static constexpr int L = L_, GW = GW_, V = V_, E = 8 * V_;
    static constexpr bool VEC = VEC_, CLUSTER = CLUSTER_;
    static constexpr int THREADS = GW == 1 ? 256 : 32 * GW;
    static constexpr int ROWS = GW == 1 ? 8 * (32 / L) : 1;        // a CTA works on at once
    static constexpr int G = GW == 1 ? L : 32 * GW;                // threads of a row in one CTA
    static constexpr int COLS = G * E;                             // columns that they hold
    static_assert(GW == 1 || L == 32, "whole warps");
};

constexpr int kNormMaxCluster = 8;
constexpr int kNormMaxWarps = 16 * kNormMaxCluster;                // of a row

__device__ __forceinline__ float norm_get(const uint16_t* p) { return bf16f(*p); }
__device__ __forceinline__ float norm_get(const float* p) { return *p; }
__device__ __forceinline__ void norm_put(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void norm_put(float* p, float v) { *p = v; }

__device__ __forceinline__ void get8(const uint16_t* p, float* v) {
    const uint4 q = ldu4(p);
    v[0] = bf16lo(q.x); v[1] = bf16hi(q.x); v[2] = bf16lo(q.y); v[3] = bf16hi(q.y);
    v[4] = bf16lo(q.z); v[5] = bf16hi(q.z); v[6] = bf16lo(q.w); v[7] = bf16hi(q.w);
}
__device__ __forceinline__ void get8(const float* p, float* v) {
    const float4 a = ld4(p), b = ld4(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void put8(uint16_t* p, const float* v) {
    stu4(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}
__device__ __forceinline__ void put8(float* p, const float* v) {
    st4(p, make_float4(v[0], v[1], v[2], v[3]));
    st4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}

// Column of a thread's element e; t: the thread's place among the G of its row, first: the
// columns before this CTA's.
template <class C>
__device__ __forceinline__ int norm_col(int first, int t, int e) {
    return first + (C::VEC ? ((e >> 3) * C::G + t) * 8 + (e & 7) : e * C::G + t);
}

// A thread's elements of a row; 0 past its end.
template <class C, typename T>
__device__ __forceinline__ void norm_load(const T* row, int cols, int first, int t, float (&v)[C::E]) {
    if constexpr (C::VEC) {
#pragma unroll
        for (int c = 0; c < C::V; ++c) {
            const int at = norm_col<C>(first, t, 8 * c);
            if (at + 8 <= cols) {
                get8(row + at, v + 8 * c);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[8 * c + k] = at + k < cols ? norm_get(row + at + k) : 0.f;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int at = norm_col<C>(first, t, e);
            v[e] = at < cols ? norm_get(row + at) : 0.f;
        }
    }
}
template <class C, typename T>
__device__ __forceinline__ void norm_store(T* row, int cols, int first, int t, const float (&v)[C::E]) {
    if constexpr (C::VEC) {
#pragma unroll
        for (int c = 0; c < C::V; ++c) {
            const int at = norm_col<C>(first, t, 8 * c);
            if (at + 8 <= cols) {
                put8(row + at, v + 8 * c);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (at + k < cols) norm_put(row + at + k, v[8 * c + k]);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < C::E; ++e) {
            const int at = norm_col<C>(first, t, e);
            if (at < cols) norm_put(row + at, v[e]);
        }
    }
}
// A vector of one row's width that may start at any element; `fill` where it is not there.
template <class C, typename T>
__device__ __forceinline__ void norm_vector(const T* p, int cols, int first, int t, float fill, float (&v)[C::E]) {
#pragma unroll
    for (int e = 0; e < C::E; ++e) {
        const int at = norm_col<C>(first, t, e);
        v[e] = p && at < cols ? norm_get(p + at) : p ? 0.f : fill;
    }
}

// Sums over a row, the same bits in each of its threads.  buf: float[2][NV][kNormMaxWarps] of
// shared memory where a row has more than one warp; the two halves take turns, so that one
// barrier per sum is enough.
template <class C, int NV>
struct RowSum {
    float* buf;
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&s)[NV], int warp, int lane, int n_ctas) {
        constexpr int W = C::GW == 1 ? C::L : 32;
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
        if constexpr (C::GW > 1) {
            float* const b = buf + turn * NV * kNormMaxWarps;
            if constexpr (C::CLUSTER) {
                if (lane < n_ctas) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        st_cluster(map_rank(smem_addr(b + i * kNormMaxWarps + int(cluster_rank()) * C::GW + warp), lane), s[i]);
                }
                __syncwarp();
                cluster_arrive();
                cluster_wait();
            } else {
                if (lane == 0) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) b[i * kNormMaxWarps + warp] = s[i];
                }
                __syncthreads();
            }
            const int n = C::CLUSTER ? C::GW * n_ctas : C::GW;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float t = 0.f;
                for (int w = 0; w < n; w += 4) {
                    const float4 q = ld4(b + i * kNormMaxWarps + w);
                    t += (q.x + q.y) + (q.z + q.w);
                }
                s[i] = t;
            }
            turn ^= 1;
        }
    }
};

// The configuration of a width: f(cfg) for the narrowest that holds it.
template <typename T, bool VEC, class F>
cudaError_t norm_dispatch(int64_t cols, F&& f) {
    if (cols <= 32) return f(NormCfg<T, 4, 1, 1, VEC>{});
    if (cols <= 64) return f(NormCfg<T, 8, 1, 1, VEC>{});
    if (cols <= 128) return f(NormCfg<T, 16, 1, 1, VEC>{});
    if (cols <= 256) return f(NormCfg<T, 32, 1, 1, VEC>{});
    if (cols <= 512) return f(NormCfg<T, 32, 1, 2, VEC>{});
    if (cols <= 1024) return f(NormCfg<T, 32, 1, 4, VEC>{});
    if (cols <= 2048) return f(NormCfg<T, 32, 4, 2, VEC>{});
    if (cols <= 4096) return f(NormCfg<T, 32, 8, 2, VEC>{});
    if (cols <= 8192) return f(NormCfg<T, 32, 16, 2, VEC>{});
    return f(NormCfg<T, 32, 16, 2, VEC, true>{});
}

// CTAs of a row (a cluster where there are more than one).
template <class C>
int norm_ctas(int64_t cols) {
    if (!C::CLUSTER) return 1;
    int n = 2;
    while (int64_t(n) * C::COLS < cols) n *= 2;
    return n;
}

template <typename... KArgs, typename... Args>
cudaError_t norm_launch(void (*kernel)(KArgs...), int groups, int ctas, int threads, size_t smem, cudaStream_t st, Args&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * ctas));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

}  // namespace
}  // namespace fsdp
