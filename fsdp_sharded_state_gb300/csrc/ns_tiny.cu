// ns_tiny.cu -- Newton-Schulz steps of small matrices, a CTA for each from its norm to its result.
//
// What bounds small matrices on the products' kernels is their 17 launches of 5 us, each for a
// microsecond of work in one tile.  Here X, A and B stay in shared memory as fp32 and the FMA units form
// the products, with a barrier in place of a launch.
//
// What bounds it then is reading shared memory, so a thread adds up 4 x 4 elements of a product, both
// operands 16 bytes at a time, two fp32 per instruction: rows of X by rows of X (A = X X^T, and A A, since A
// is symmetric; tiles at or below the diagonal), or rows of B by four columns of X.  Where a product
// has fewer such tiles than the CTA has threads, neighbouring lanes share out k and hand each other
// the parts of the sums that each is to keep.  64 x 32 takes 17 us, 64 x 64 47 us (2 x 2 elements a
// thread: 24 and 68).
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "ns.hpp"

namespace fsdp {
namespace {

constexpr int kTinyThreads = 512;
constexpr int64_t kTinySide = 124;              // its 496 tiles are a thread each
constexpr int64_t kTinySmem = 220 * 1024;
// m^2 (3 n / 2 + m), a step's multiplications: above, one SM takes longer than the products' kernels
// do for matrices of up to 256 x 256, 85 to 90 us (64 x 120, 1.0 million: 62 us; 64 x 256, 1.8: 106;
// 96 x 96, 2.2: 122).
constexpr int64_t kTinyWork = 1450000;

struct TinySteps {
    float f[kNsMaxSteps][3];
    int32_t steps;
};

// Sizes of a matrix in shared memory: the sides padded with zeros to multiples of four, and row
// strides at which the lanes that read neighbouring rows (and, `slices` of them, neighbouring 16
// bytes) meet no bank twice.
struct TinyShape {
    int m, n, mp, np, ldx, lda;
    int gram, step;                             // lanes that share out k
};
__host__ __device__ inline int pad4(int n) { return (n + 3) / 4 * 4; }
__host__ __device__ inline int tiny_ld(int n, int slices) {
    const int want = slices >= 8 ? 1 : slices;  // 16-byte units, modulo 8
    int units = n / 4;
    while (units % 8 != want) ++units;
    return 4 * units;
}
TinyShape tiny_shape(int64_t m, int64_t n) {
    TinyShape s;
    s.m = int(m);
    s.n = int(n);
    s.mp = pad4(s.m);
    s.np = pad4(s.n);
    const int q = s.mp / 4, low = q * (q + 1) / 2, all = q * (s.np / 4);
    s.gram = s.step = 1;
    while (s.gram < 8 && 2 * s.gram * low <= kTinyThreads && 2 * s.gram <= s.mp / 4) s.gram *= 2;
    while (s.step < 8 && 2 * s.step * all <= kTinyThreads && 2 * s.step <= s.mp / 4) s.step *= 2;
    s.ldx = tiny_ld(s.np, s.gram);
    s.lda = tiny_ld(s.mp, s.gram);
    return s;
}

__device__ __forceinline__ float tiny_get(const void* p, int64_t i, int bf16) {
    return bf16 ? bf16f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t make_pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ ulonglong2 two_pairs(const float* p) { return *reinterpret_cast<const ulonglong2*>(p); }

// A thread's place in the products, the same in every step: its tile (rows i + e q) and its slice of k.
struct TinyPlace {
    int i, j, slice;
    bool have;
};
__device__ __forceinline__ TinyPlace gram_place(int q, int slices, int tid) {
    TinyPlace p;
    const int tile = tid / slices;
    p.slice = tid % slices;
    p.have = tile < q * (q + 1) / 2;
    int i = int((sqrtf(8.f * float(tile) + 1.f) - 1.f) * 0.5f);
    if (i * (i + 1) / 2 > tile) --i;
    if ((i + 1) * (i + 2) / 2 <= tile) ++i;
    p.i = p.have ? i : 0;
    p.j = p.have ? tile - i * (i + 1) / 2 : 0;
    return p;
}

// f(r, c, v) and, from tiles off the diagonal, f(c, r, v), with v the sum over k of row r times row c.
// Tile (i, j) has rows i + e q and columns j + f q, so that neighbouring tiles read neighbouring rows.
template <int S, class F>
__device__ __forceinline__ void tiny_gram(const float* x, int ld, int q, int kp, const TinyPlace& at, F&& f) {
    const int i = at.i, j = at.j, slice = at.slice;
    const float *const a = x + i * ld, *const b = x + j * ld;
    const int side = q * ld;
    uint64_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = 0;
#pragma unroll 1
    for (int k = 4 * slice; k < kp; k += 4 * S) {
        ulonglong2 u[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[e] = two_pairs(a + e * side + k);
            v[e] = two_pairs(b + e * side + k);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int g = 0; g < 4; ++g) p[4 * e + g] = fma_pair(u[e].y, v[g].y, fma_pair(u[e].x, v[g].x, p[4 * e + g]));
    }
    float s[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 h = halves(p[e]);
        s[e] = h.x + h.y;
    }
    // lane by lane halves of the sums change hands: lane `slice` keeps 16 / S of them, from `first` on
    int first = 0;
#pragma unroll
    for (int round = 0; round < 4; ++round) {
        const int bit = 1 << round, n = 8 >> round;
        if (bit >= S) break;
        const bool up = slice & bit;
        first += up ? n : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e >= n) break;
            const float mine = up ? s[e + n] : s[e], other = up ? s[e] : s[e + n];
            s[e] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
        }
    }
    if (!at.have) return;
#pragma unroll
    for (int e = 0; e < 16 / S; ++e) {
        const int r = i + (first + e) / 4 * q, c = j + (first + e) % 4 * q;
        f(r, c, s[e]);
        if (i != j) f(c, r, s[e]);
    }
}

// y = a x + b x: rows i + e q, columns 4 j on; `first`: the thread's first tile.
template <int S>
__device__ __forceinline__ void tiny_step(const float* x, float* y, const float* b, float fa, const TinyShape& sh, const TinyPlace& at,
                                          int tid) {
    const int q = sh.mp / 4, wide = sh.np / 4, tiles = q * wide, slice = at.slice;
    for (int base = 0; base < tiles; base += kTinyThreads / S) {
        int i = at.i, j = at.j;
        bool have = at.have;
        if (base > 0) {
            const int tile = base + tid / S;
            have = tile < tiles;
            i = have ? tile / wide : 0;
            j = have ? tile % wide * 4 : 0;
        }
        uint64_t s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0;
#pragma unroll 1
        for (int l = 4 * slice; l < sh.mp; l += 4 * S) {
            float4 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const float4*>(b + (i + e * q) * sh.lda + l);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const ulonglong2 v = two_pairs(x + (l + d) * sh.ldx + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = d == 0 ? w[e].x : d == 1 ? w[e].y : d == 2 ? w[e].z : w[e].w;
                    const uint64_t ff = make_pair(f, f);
                    s[2 * e] = fma_pair(ff, v.x, s[2 * e]);
                    s[2 * e + 1] = fma_pair(ff, v.y, s[2 * e + 1]);
                }
            }
        }
        int first = 0;
#pragma unroll
        for (int round = 0; round < 3; ++round) {
            const int bit = 1 << round, n = 4 >> round;
            if (bit >= S) break;
            const bool up = slice & bit;
            first += up ? n : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e >= n) break;
                const uint64_t mine = up ? s[e + n] : s[e], other = up ? s[e] : s[e + n];
                s[e] = add_pair(mine, __shfl_xor_sync(0xffffffffu, other, bit));
            }
        }
        if (!have) continue;
        const uint64_t aa = make_pair(fa, fa);
#pragma unroll
        for (int e = 0; e < 8 / S; ++e) {
            const int at = (i + (first + e) / 2 * q) * sh.ldx + j + (first + e) % 2 * 2;
            *reinterpret_cast<uint64_t*>(y + at) = fma_pair(aa, *reinterpret_cast<const uint64_t*>(x + at), s[e]);
        }
    }
}

template <int GRAM, int STEP>
__global__ void __launch_bounds__(kTinyThreads, 1)
k_ns_tiny(const __grid_constant__ NsMatrices src, const __grid_constant__ NsMatrices dst, const TinyShape sh, float eps,
          const __grid_constant__ TinySteps st) {
    extern __shared__ __align__(16) float tiny_smem[];
    __shared__ float part[kTinyThreads / 32];
    const int tid = threadIdx.x, mat = blockIdx.x;
    float *x = tiny_smem, *y = x + sh.mp * sh.ldx, *const a = y + sh.mp * sh.ldx, *const b = a + sh.mp * sh.lda;
    for (int i = tid; i < sh.mp * (sh.ldx + sh.lda) / 2; i += kTinyThreads) reinterpret_cast<float4*>(tiny_smem)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    pdl_wait();
    // the matrix, its longer side along x's rows, and its sum of squares
    const bool tall = src.tall >> mat & 1;
    const int rows = tall ? sh.n : sh.m, cols = tall ? sh.m : sh.n;
    float square = 0.f, lost = 0.f;
    for (int i = tid; i < rows * cols; i += kTinyThreads) {
        const int r = i / cols, c = i - r * cols;
        const float v = tiny_get(src.p[mat], r * src.ld[mat] + c, src.bf16);
        x[tall ? c * sh.ldx + r : r * sh.ldx + c] = v;
        add_carefully(__fmul_rn(v, v), square, lost);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
    if ((tid & 31) == 0) part[tid >> 5] = square;
    __syncthreads();
    square = 0.f;
#pragma unroll
    for (int k = 0; k < kTinyThreads / 32; ++k) square += part[k];
    const float norm = sqrtf(square), factor = 1.f / (norm < eps ? eps : norm);          // a NaN stays
    for (int i = tid; i < sh.mp * sh.ldx; i += kTinyThreads) x[i] *= factor;
    __syncthreads();
    const int lda = sh.lda, q = sh.mp / 4;
    const TinyPlace pg = gram_place(q, GRAM, tid);
    TinyPlace ps;
    {
        const int wide = sh.np / 4, tile = tid / STEP;
        ps.slice = tid % STEP;
        ps.have = tile < q * wide;
        ps.i = ps.have ? tile / wide : 0;
        ps.j = ps.have ? tile % wide * 4 : 0;
    }
    for (int k = 0; k < st.steps; ++k) {
        const float fa = st.f[k][0], fb = st.f[k][1], fc = st.f[k][2];
        tiny_gram<GRAM>(x, sh.ldx, q, sh.np, pg, [&](int r, int c, float v) { a[r * lda + c] = v; });
        __syncthreads();
        tiny_gram<GRAM>(a, lda, q, sh.mp, pg, [&](int r, int c, float v) { b[r * lda + c] = __fmaf_rn(fc, v, __fmul_rn(fb, a[r * lda + c])); });
        __syncthreads();
        tiny_step<STEP>(x, y, b, fa, sh, ps, tid);
        __syncthreads();
        float* const z = x;
        x = y;
        y = z;
    }
    for (int i = tid; i < rows * cols; i += kTinyThreads) {
        const int r = i / cols, c = i - r * cols;
        const float v = x[tall ? c * sh.ldx + r : r * sh.ldx + c];
        const int64_t at = r * dst.ld[mat] + c;
        if (dst.bf16) static_cast<uint16_t*>(dst.p[mat])[at] = to_bf16(v);
        else static_cast<float*>(dst.p[mat])[at] = v;
    }
}

size_t tiny_bytes(const TinyShape& s) { return size_t(2 * s.mp) * size_t(s.ldx + s.lda) * 4; }

template <int GRAM, int STEP>
cudaError_t launch_tiny(const NsMatrices& src, const NsMatrices& dst, int batch, const TinyShape& sh, float eps, const TinySteps& s,
                        cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    static std::atomic<uint64_t> prepared{0};
    if (e == cudaSuccess && (dev >= 64 || !(prepared.load(std::memory_order_relaxed) >> dev & 1))) {
        e = cudaFuncSetAttribute(k_ns_tiny<GRAM, STEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTinySmem));
        if (e == cudaSuccess && dev < 64) prepared.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    return e == cudaSuccess ? launch(k_ns_tiny<GRAM, STEP>, dim3(unsigned(batch)), dim3(kTinyThreads), tiny_bytes(sh), st, src, dst, sh, eps, s)
                            : e;
}

}  // namespace

bool use_ns_tiny(int64_t m, int64_t n) {
    return m <= kTinySide && n < (1 << 16) && m * m * (3 * n / 2 + m) <= kTinyWork && tiny_bytes(tiny_shape(m, n)) <= size_t(kTinySmem);
}

cudaError_t launch_ns_tiny(const NsMatrices& src, const NsMatrices& dst, int batch, int64_t m, int64_t n, float eps, const float* coeffs,
                           int steps, const float* usual, cudaStream_t st) {
    TinySteps s = {};
    s.steps = steps;
    for (int k = 0; k < steps; ++k)
        for (int i = 0; i < 3; ++i) s.f[k][i] = coeffs ? coeffs[3 * k + i] : usual[i];
    const TinyShape sh = tiny_shape(m, n);
    auto step = [&](auto gram) {
        constexpr int G = decltype(gram)::value;
        switch (sh.step) {
            case 1: return launch_tiny<G, 1>(src, dst, batch, sh, eps, s, st);
            case 2: return launch_tiny<G, 2>(src, dst, batch, sh, eps, s, st);
            case 4: return launch_tiny<G, 4>(src, dst, batch, sh, eps, s, st);
            default: return launch_tiny<G, 8>(src, dst, batch, sh, eps, s, st);
        }
    };
    switch (sh.gram) {
        case 1: return step(std::integral_constant<int, 1>{});
        case 2: return step(std::integral_constant<int, 2>{});
        case 4: return step(std::integral_constant<int, 4>{});
        default: return step(std::integral_constant<int, 8>{});
    }
}

}  // namespace fsdp
