// norm_rows.cuh -- what the layer-norm kernels share: how a row is spread over threads, its
// loads and stores, and sums over it.
//
// A row belongs to a group of threads that hold it in registers from its load to its store:
// L lanes of a warp (up to 512 columns; a warp then works on 32 / L rows at once), GW warps of a CTA
// (up to 8192, in forward 16384), or GW warps in each CTA of a cluster (up to 65536).  A thread holds 8 V columns:
// chunks of 16 bytes where rows are made of whole ones (VEC), else single columns that are a
// group's width apart, so that a warp's accesses are contiguous either way.
//
// Rows come through shared memory (RowRing): loads of a row by the threads that wait for it
// leave HBM idle from its last byte to the next row's request (16384 x 4096 bf16 forward 121 us, 0.33 of the
// copy rate); bulk copies of the next rows run while one is worked on, whatever the registers hold
// (79 us).  What then bounds a wide row is the issue of its instructions, so elements are worked on in
// pairs (add, mul and fma of two fp32 at once, each rounded as its single form), rows are read from
// shared memory by address, and what can be formed once a stage is (46 us, 0.86 of the copy rate).  Single
// columns issue more than chunks do: 8192 x 4097 bf16 forward takes 56 us where 8192 x 5120 takes 35.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.hpp"
#include "norm.hpp"
#include "tc5.cuh"

namespace fsdp {
namespace {

template <typename T_, int L_, int GW_, int V_, bool VEC_, bool CLUSTER_ = false>
struct NormCfg {
    using T = T_;
    static constexpr int L = L_, GW = GW_, V = V_, E = 8 * V_;
    static constexpr int W = 16 / sizeof(T);                       // columns of a chunk
    static constexpr bool VEC = VEC_, CLUSTER = CLUSTER_;
    static constexpr int P = E / 2;                                // pairs of a thread
    static constexpr int THREADS = GW <= 8 ? 256 : 32 * GW;
    static constexpr int SIDE = THREADS / (32 * GW);               // groups side by side in a CTA
    static constexpr int G = GW == 1 ? L : 32 * GW;                // threads of a row in one CTA
    static constexpr int COLS = G * E;                             // columns that they hold
    static_assert(GW == 1 || L == 32, "whole warps");
    static_assert(GW <= 2 || GW % 4 == 0, "sums of warps, four at a time");
};

constexpr int kNormMaxWarps = 16 * 8;                              // of a row, in a cluster of 8

__device__ __forceinline__ float norm_get(const uint16_t* p) { return bf16f(*p); }
__device__ __forceinline__ float norm_get(const float* p) { return *p; }
__device__ __forceinline__ void norm_put(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void norm_put(float* p, float v) { *p = v; }

// ---- two fp32 in a register pair -------------------------------------------------------
using pair = uint64_t;
__device__ __forceinline__ pair pair_of(float a, float b) {
    pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(pair p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ pair add2(pair a, pair b) {
    pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair mul2(pair a, pair b) {
    pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair fma2(pair a, pair b, pair c) {
    pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float both(pair p) {
    const float2 f = split(p);
    return f.x + f.y;
}

// A chunk of 16 bytes as pairs.
__device__ __forceinline__ void norm_get16(const uint16_t* p, pair* v) {
    const uint4 q = ldu4(p);
    v[0] = pair_of(bf16lo(q.x), bf16hi(q.x));
    v[1] = pair_of(bf16lo(q.y), bf16hi(q.y));
    v[2] = pair_of(bf16lo(q.z), bf16hi(q.z));
    v[3] = pair_of(bf16lo(q.w), bf16hi(q.w));
}
__device__ __forceinline__ void norm_get16(const float* p, pair* v) {
    const float4 a = ld4(p);
    v[0] = pair_of(a.x, a.y);
    v[1] = pair_of(a.z, a.w);
}
// The same from shared memory, by address.
__device__ __forceinline__ void smem_get16(uint32_t p, pair* v, const uint16_t*) {
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(p) : "memory");
    v[0] = pair_of(bf16lo(q.x), bf16hi(q.x));
    v[1] = pair_of(bf16lo(q.y), bf16hi(q.y));
    v[2] = pair_of(bf16lo(q.z), bf16hi(q.z));
    v[3] = pair_of(bf16lo(q.w), bf16hi(q.w));
}
__device__ __forceinline__ void smem_get16(uint32_t p, pair* v, const float*) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(p) : "memory");
}
__device__ __forceinline__ float smem_get(uint32_t p, const uint16_t*) {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(p) : "memory");
    return bf16f(h);
}
__device__ __forceinline__ float smem_get(uint32_t p, const float*) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(p) : "memory");
    return f;
}
__device__ __forceinline__ uint32_t pack_pair(pair p) {
    const float2 f = split(p);
    return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ void norm_put16(uint16_t* p, const pair* v) {
    stu4(p, make_uint4(pack_pair(v[0]), pack_pair(v[1]), pack_pair(v[2]), pack_pair(v[3])));
}
__device__ __forceinline__ void norm_put16(float* p, const pair* v) {
    const float2 a = split(v[0]), b = split(v[1]);
    st4(p, make_float4(a.x, a.y, b.x, b.y));
}

// Column of a thread's element e; t: the thread's place among the G of its row, first: the
// columns before this CTA's.
template <class C>
__device__ __forceinline__ int norm_col(int first, int t, int e) {
    return first + (C::VEC ? ((e / C::W) * C::G + t) * C::W + e % C::W : e * C::G + t);
}

// Whether all of a thread's columns are in the row.
template <class C>
__device__ __forceinline__ bool norm_full(int cols, int first, int t) {
    return norm_col<C>(first, t, C::E - 1) < cols;
}

// Elements past the row's end made 0.  Chunks are in it or past it as a whole: tested element by
// element, 4096 x 10000 bf16 forward took 150 us.
template <class C>
__device__ __forceinline__ void norm_trim(int cols, int first, int t, pair (&v)[C::P]) {
#pragma unroll
    for (int e = 0; e < C::E; e += 2) {
        const float2 f = split(v[e / 2]);
        const bool in = norm_col<C>(first, t, C::VEC ? e / C::W * C::W : e) < cols;
        v[e / 2] = pair_of(in ? f.x : 0.f, (C::VEC ? in : norm_col<C>(first, t, e + 1) < cols) ? f.y : 0.f);
    }
}

// A thread's elements of a row whose column `first` is at `row` in shared memory; 0 past its end,
// where the thread is not full.  (Full threads have code of their own, here and below: with tests, even of a
// bit, between the loads of the chunks, 16384 x 4096 bf16 backward took 123 us instead of 77.)
template <class C>
__device__ __forceinline__ void norm_load(uint32_t row, int cols, int first, int t, bool full, pair (&v)[C::P]) {
    using T = typename C::T;
    constexpr const T* type = nullptr;
    constexpr int S = int(sizeof(T));
    auto at_or_0 = [&](int e) { return norm_col<C>(first, t, e) < cols ? smem_get(row + uint32_t(norm_col<C>(0, t, e) * S), type) : 0.f; };
    if (C::VEC && full) {
#pragma unroll
        for (int c = 0; c < C::E; c += C::W) smem_get16(row + uint32_t(norm_col<C>(0, t, c) * S), v + c / 2, type);
    } else if (C::VEC) {                         // for chunks past the row's end its first
#pragma unroll
        for (int c = 0; c < C::E; c += C::W) smem_get16(norm_col<C>(first, t, c) < cols ? row + uint32_t(norm_col<C>(0, t, c) * S) : row, v + c / 2, type);
        norm_trim<C>(cols, first, t, v);
    } else if (full) {
#pragma unroll
        for (int e = 0; e < C::E; e += 2)
            v[e / 2] = pair_of(smem_get(row + uint32_t(norm_col<C>(0, t, e) * S), type), smem_get(row + uint32_t(norm_col<C>(0, t, e + 1) * S), type));
    } else {
#pragma unroll
        for (int e = 0; e < C::E; e += 2) v[e / 2] = pair_of(at_or_0(e), at_or_0(e + 1));
    }
}
// And into a row of a matrix in global memory.
template <class C, typename T>
__device__ __forceinline__ void norm_store(T* row, int cols, int first, int t, bool full, const pair (&v)[C::P]) {
    T* const p = row + norm_col<C>(first, t, 0);
    auto put = [&](int e) {
        const float2 f = split(v[e / 2]);
        norm_put(p + norm_col<C>(0, 0, e), e & 1 ? f.y : f.x);
    };
    auto in = [&](int e) { return norm_col<C>(first, t, e) < cols; };
    if (C::VEC && full) {
#pragma unroll
        for (int c = 0; c < C::E; c += C::W) norm_put16(p + norm_col<C>(0, 0, c), v + c / 2);
    } else if (C::VEC) {
#pragma unroll
        for (int c = 0; c < C::E; c += C::W)
            if (in(c)) norm_put16(p + norm_col<C>(0, 0, c), v + c / 2);
    } else if (full) {
#pragma unroll
        for (int e = 0; e < C::E; ++e) put(e);
    } else {
#pragma unroll
        for (int e = 0; e < C::E; ++e)
            if (in(e)) put(e);
    }
}
// A vector of one row's width that may start at any element; `fill` where it is not there.
template <class C, typename T>
__device__ __forceinline__ void norm_vector(const T* p, int cols, int first, int t, float fill, pair (&v)[C::P]) {
    auto get = [&](int e) {
        const int at = norm_col<C>(first, t, e);
        return p && at < cols ? norm_get(p + at) : p ? 0.f : fill;
    };
    if constexpr (C::VEC) {
        if (p && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && norm_full<C>(cols, first, t)) {
#pragma unroll
            for (int c = 0; c < C::E; c += C::W) norm_get16(p + norm_col<C>(first, t, c), v + c / 2);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < C::E; e += 2) v[e / 2] = pair_of(get(e), get(e + 1));
}

// The threads of a group that is more than a warp, and no others of the CTA.
template <class C>
__device__ __forceinline__ void group_sync(int group) {
    if constexpr (C::SIDE == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * C::GW) : "memory");
}

// Sums over a row, the same bits in each of its threads.  Where a row has more than one warp, buf is
// FLOATS of shared memory for each group; its two halves take turns, so that one barrier per
// sum is enough: a warp sends into a half again once it has had the sum between, to which every
// warp gave its part after it had used the half.
//
// A cluster's warps send their parts to each of its CTAs, where they are counted on a barrier (two
// of them at `bars`, for the halves).  A barrier of the cluster waits for the stores to global
// memory before it as well: with that, 4096 x 16384 bf16 backward took 137 us.
template <class C, int NV>
struct RowSum {
    static constexpr int WARPS = C::CLUSTER ? kNormMaxWarps : C::GW < 4 ? 4 : C::GW;
    static constexpr int FLOATS = 2 * NV * WARPS;
    float* buf;
    uint32_t bars;
    uint64_t wait_ns;
    int turn = 0;
    uint32_t phases = 0;
    __device__ __forceinline__ void operator()(float (&s)[NV], int warp, int lane, int n_ctas) {
        constexpr int W = C::GW == 1 ? C::L : 32;
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
        if constexpr (C::GW > 1) {
            const int mine = warp % C::GW, group = warp / C::GW;
            float* const b = buf + group * FLOATS + turn * NV * WARPS;
            if constexpr (C::CLUSTER) {
                const uint32_t bar = bars + 8 * turn;
                __syncwarp();                    // before the sends, all lanes' reads of the stage that they let another thread fill again
                if (mine == 0 && lane == 0) mbar_arrive_tx(bar, uint32_t(4 * NV * C::GW * n_ctas));
                if (lane < n_ctas) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        st_cluster_tx(map_rank(smem_addr(b + i * WARPS + int(cluster_rank()) * C::GW + mine), lane), s[i], map_rank(bar, lane));
                }
                __syncwarp();
                if (!mbar_wait_bounded(bar, phases >> turn & 1, wait_ns)) {
                    wait_ns = 0;
                    atomicOr(&g_wait_error, 1u);
                }
                phases ^= 1u << turn;
            } else {
                if (lane == 0) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) b[i * WARPS + mine] = s[i];
                }
                group_sync<C>(group);
            }
            const int n = C::CLUSTER ? C::GW * n_ctas : C::GW;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (C::GW == 2) {
                    s[i] = b[i * WARPS] + b[i * WARPS + 1];
                } else {
                    float t = 0.f;
#pragma unroll 4
                    for (int w = 0; w < n; w += 4) {
                        const float4 q = ld4(b + i * WARPS + w);
                        t += (q.x + q.y) + (q.z + q.w);
                    }
                    s[i] = t;
                }
            }
            turn ^= 1;
        }
    }
};

// A CTA's ring of stages in shared memory that bulk copies fill with the next rows: `block` rows for
// each of its groups, or its share of one row; per matrix the 16-byte granules that hold them, as one
// piece where the rows are back to back, else a piece a row.  Rows may start at any element: the
// bytes around a piece, which are in its own granules, are read and not used.  Stages are large, since
// a copy takes some 65 ns of the copy engine beside 22 ns a KB: with 2 KB for each warp apart, 65536 x 256
// backward without sums took 36 us.  The group that is last to have read a stage fills it again.
//
// Waits are bounded: after one that gave up, which is recorded for fsdp_check_status, the others
// give up at once, and the threads go through their rows with what the stages hold.
constexpr int kRingStages = 8;
constexpr int kRingFront = 256;                  // the stages' barriers and counts, the barriers of a cluster's sums, the matrices' places
constexpr int kRingSums = 12 * kRingStages, kRingPlaces = 128;

// Bytes of a row's piece.
__host__ __device__ inline int ring_piece(int cols, int esize) { return (cols * esize + 15) / 16 * 16 + 16; }

template <class C, int N>
struct RowRing {
    using T = typename C::T;
    static constexpr bool PLACES = C::SIDE > 1 && N > 1;
    // Of this CTA's columns.  PLACES: read from shared memory, by the warp that copies, instead of from
    // 12 registers that backward's kernels miss.
    const T* base[N];
    int64_t ld[N];
    bool there[N];                               // the last may not be
    uint32_t front, at;                          // the ring in shared memory, and its present stage
    uint32_t rows, step;                         // of all, and between a CTA's stages
    int stages, most, piece, cols;               // most: rows of a stage; cols: of this CTA
    uint32_t between[N];                         // bytes from a row of a stage to the next
    uint32_t low[N], low_step[N], low_row[N];    // rows of any alignment: the first's address mod 16, and what to add for the next stage's and row's
    bool back[N];                                // rows back to back
    uint64_t wait_ns;
    int s = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ RowRing(unsigned char* smem, int first, int all, int stages_, int block, uint32_t rows_, uint32_t step_, uint64_t wait)
        : front(smem_addr(smem)), at(smem_addr(smem) + kRingFront), rows(rows_), step(step_), stages(stages_), most(C::SIDE * block), wait_ns(wait) {
        const int left = all - first;
        cols = left < 0 ? 0 : left < C::COLS ? left : C::COLS;
        piece = ring_piece(all < C::COLS ? all : C::COLS, int(sizeof(T)));
    }
    __device__ __forceinline__ void matrix(int k, const void* p, int64_t ld_, int first, uint32_t row0) {
        base[k] = static_cast<const T*>(p) + first;
        ld[k] = ld_;
        there[k] = p != nullptr;
        back[k] = C::SIDE > 1 && ld_ == cols;
        between[k] = back[k] ? uint32_t(cols) * uint32_t(sizeof(T)) : uint32_t(piece);
        if constexpr (!C::VEC) {
            low_row[k] = uint32_t(ld_) * uint32_t(sizeof(T));
            low_step[k] = step * low_row[k];
            low[k] = uint32_t(reinterpret_cast<uintptr_t>(base[k])) + row0 * low_row[k];
        }
    }
    __device__ __forceinline__ uint32_t bar(int i) const { return front + 8 * i; }
    __device__ __forceinline__ uint32_t count(int i) const { return front + 8 * kRingStages + 4 * i; }
    __device__ __forceinline__ uint32_t sums(int i) const { return front + kRingSums + 16 * i; }
    // By one thread, before any other uses the ring.
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < stages; ++i) {
            mbar_init(bar(i), 1);
            asm volatile("st.shared.u32 [%0], 0;" ::"r"(count(i)) : "memory");
        }
        if constexpr (PLACES) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(front + kRingPlaces + 16 * k), "l"(base[k]), "l"(ld[k]) : "memory");
        }
        for (int i = 0; C::CLUSTER && i < 4; ++i) mbar_init(sums(i / 2) + 8 * (i & 1), 1);
        mbar_fence_init();
    }
    // n rows from `row` on of matrix k to `dst`; counts the bytes, copies where told to.
    __device__ __forceinline__ void copy(uint32_t row, int n, uint32_t dst, int k, int i, uint32_t& bytes, bool issue) const {
        const T* p = base[k];
        int64_t l = ld[k];
        if constexpr (PLACES) asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(p), "=l"(l) : "r"(front + kRingPlaces + 16 * k) : "memory");
        const uintptr_t a = reinterpret_cast<uintptr_t>(p + row * l);
        const uint32_t size = cols > 0 ? uint32_t((a & 15) + int64_t(n) * cols * int64_t(sizeof(T)) + 15) & ~15u : 0;   // a cluster's CTA past the row's end
        bytes += size;
        if (issue && size) bulk_g2s(dst, reinterpret_cast<const void*>(a & ~uintptr_t(15)), size, bar(i));
    }
    // The rows from `row` on into stage i: by one thread (SIDE = 1) or one warp.
    __device__ __forceinline__ void fetch(uint32_t row, int i, int lane) const {
        const int n = rows - row < uint32_t(most) ? int(rows - row) : most;
        const uint32_t to = front + kRingFront + uint32_t(i * N * most * piece);
        if constexpr (C::SIDE == 1 && C::VEC) {  // the thread that does this is one of those that wait for each other
            const uint32_t size = (uint32_t(cols) * uint32_t(sizeof(T)) + 15) & ~15u;
            const int have = there[N - 1] ? N : N - 1;
            mbar_arrive_tx(bar(i), uint32_t(have) * size);
#pragma unroll
            for (int k = 0; k < N; ++k)          // size 0: a cluster's CTA past the row's end
                if (k < have && size) bulk_g2s(to + uint32_t(k * piece), base[k] + row * ld[k], size, bar(i));
            return;
        }
        bool all = true;
#pragma unroll
        for (int k = 0; k < N; ++k) all = all && (C::SIDE == 1 || !there[k] || back[k]);
        if (all) {
            if (C::SIDE > 1 && lane != 0) return;
            uint32_t bytes = 0;
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (there[k]) copy(row, n, 0, k, i, bytes, false);
            mbar_arrive_tx(bar(i), bytes);
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (there[k]) copy(row, n, to + uint32_t(k * most * piece), k, i, bytes, true);
            return;
        }
        // the lanes share out the rows of the matrices whose rows are apart
        uint32_t bytes = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (!there[k]) continue;
            const bool w = back[k];
            for (int j = lane; j < (w ? 1 : n); j += 32) copy(row + j, w ? n : 1, 0, k, i, bytes, false);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, o);
        if (lane == 0) mbar_arrive_tx(bar(i), bytes);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (!there[k]) continue;
            const bool w = back[k];
            for (int j = lane; j < (w ? 1 : n); j += 32) copy(row + j, w ? n : 1, to + uint32_t((k * most + j) * piece), k, i, bytes, true);
        }
    }
    // The first stages; by the threads that fetch takes.
    __device__ __forceinline__ void begin(uint32_t row, int lane) const {
        for (int i = 0; i < stages; ++i)
            if (row + i * step < rows) fetch(row + i * step, i, lane);
    }
    // Where the stage holds its j-th row of matrix k: the shared-memory address of this CTA's first column.
    __device__ __forceinline__ uint32_t row_of(int j, int k) const {
        uint32_t p = at + uint32_t(k * most * piece);
        if constexpr (C::SIDE > 1) p += uint32_t(j) * between[k];
        if constexpr (!C::VEC) p += (back[k] ? low[k] : low[k] + uint32_t(j) * low_row[k]) & 15u;
        return p;
    }
    __device__ __forceinline__ void wait() {
        if (!mbar_wait_bounded(bar(s), phase, wait_ns)) {
            wait_ns = 0;
            atomicOr(&g_wait_error, 1u);
        }
    }
    // The stage that began with `row` has been read by all threads of a group, of which one warp
    // (SIDE = 1: one thread) says so.
    __device__ __forceinline__ void release(uint32_t row, int lane) const {
        row += stages * step;
        if constexpr (C::SIDE == 1) {
            if (row < rows) fetch(row, s, lane);
        } else {
            uint32_t last = 0;
            if (lane == 0) {
                __threadfence_block();
                // the last group's count goes back to 0, seen by all once the stage is full again
                asm volatile("atom.shared.inc.u32 %0, [%1], %2;" : "=r"(last) : "r"(count(s)), "r"(uint32_t(C::SIDE - 1)) : "memory");
            }
            last = __shfl_sync(0xffffffffu, last, 0);
            if (last == C::SIDE - 1 && row < rows) fetch(row, s, lane);
        }
    }
    __device__ __forceinline__ void next() {
        at += uint32_t(N * most * piece);
        if (++s == stages) {
            s = 0;
            at = front + kRingFront;
            phase ^= 1;
        }
        if constexpr (!C::VEC) {
#pragma unroll
            for (int k = 0; k < N; ++k) low[k] += low_step[k];
        }
    }
    // Before the CTA leaves: copies that were given up land within this, and no CTA sends to one that has left.
    __device__ __forceinline__ void leave(uint64_t sums_wait) const {
        if constexpr (C::CLUSTER) {
            cluster_arrive();
            cluster_wait();
        }
        if (wait_ns && sums_wait) return;
        const uint64_t t0 = global_ns();
        for (int i = 0; i < (1 << 20) && global_ns() - t0 < 2000000ull; ++i) __nanosleep(1000);
    }
};

// Host side: how many rows of a group a stage holds, how many stages, and the shared memory of a
// CTA of which per_sm share an SM.  About 8 KB of each matrix a stage, at most 32 rows a warp.
struct RingShape {
    int block, stages;
    size_t bytes;
};
template <class C>
RingShape ring_shape(int n, int64_t cols, int per_sm) {
    constexpr int es = int(sizeof(typename C::T)), side = C::GW == 1 ? 32 / C::L : 1;
    const int piece = ring_piece(int(cols < C::COLS ? cols : C::COLS), es);
    RingShape r;
    r.block = side;
    if (C::GW == 1)
        while (C::SIDE * r.block * piece < 8192 && r.block + side <= 32) r.block += side;
    const int stage = n * C::SIDE * r.block * piece, fit = (208 * 1024 / per_sm - kRingFront - 4096) / stage;
    r.stages = fit > kRingStages ? kRingStages : fit < 2 ? 2 : fit;
    r.bytes = size_t(kRingFront) + size_t(r.stages) * stage;
    return r;
}

std::atomic<bool> g_norm_launched{false};

cudaError_t take_norm_wait_error(unsigned int* flag) {
    *flag = 0;
    return g_norm_launched.load(std::memory_order_relaxed) ? take_local_wait_error(flag) : cudaSuccess;
}

int norm_sms(int dev) {
    static std::atomic<int> n[64];
    if (dev < 0 || dev >= 64) return 152;
    int v = n[dev].load(std::memory_order_relaxed);
    if (v == 0 && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) n[dev].store(v, std::memory_order_relaxed);
    return v > 0 ? v : 152;
}

// The configuration of a width: f(cfg) for the narrowest that holds it.  Backward holds six values an
// element where forward holds three: half as many columns a thread above 6144.
template <typename T, bool VEC, class F>
cudaError_t norm_dispatch_narrow(int64_t cols, F&& f) {
    if (cols <= 32) return f(NormCfg<T, 4, 1, 1, VEC>{});
    if (cols <= 64) return f(NormCfg<T, 4, 1, 2, VEC>{});
    if (cols <= 128) return f(NormCfg<T, 8, 1, 2, VEC>{});
    if (cols <= 256) return f(NormCfg<T, 16, 1, 2, VEC>{});
    if (cols <= 512) return f(NormCfg<T, 32, 1, 2, VEC>{});
    if (cols <= 1024) return f(NormCfg<T, 32, 2, 2, VEC>{});
    if (cols <= 2048) return f(NormCfg<T, 32, 4, 2, VEC>{});
    if (cols <= 4096) return f(NormCfg<T, 32, 8, 2, VEC>{});
    return f(NormCfg<T, 32, 12, 2, VEC>{});
}
constexpr int64_t kNormNarrow = 6144;
template <typename T, bool VEC, class F>
cudaError_t norm_dispatch_forward(int64_t cols, F&& f) {
    if (cols <= kNormNarrow) return norm_dispatch_narrow<T, VEC>(cols, f);
    if (cols <= 8192) return f(NormCfg<T, 32, 8, 4, VEC>{});
    if (cols <= 16384) return f(NormCfg<T, 32, 16, 4, VEC>{});
    return f(NormCfg<T, 32, 16, 2, VEC, true>{});
}
template <typename T, bool VEC, class F>
cudaError_t norm_dispatch_backward(int64_t cols, F&& f) {
    if (cols <= kNormNarrow) return norm_dispatch_narrow<T, VEC>(cols, f);
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

// The most dynamic shared memory that a kernel may ask for, set once per device.
template <typename K>
cudaError_t norm_prepare(K kernel, std::atomic<uint64_t>& done, int dev) {
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
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
    g_norm_launched.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

}  // namespace
}  // namespace fsdp
