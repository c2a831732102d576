// ns_tiny.cu -- Newton-Schulz steps of small matrices, a CTA for each from its norm to its result.
//
// What bounds small matrices on the products' kernels is their 17 launches of 5 us, each for a
// microsecond of work in one tile.  Here X, A and B stay in shared memory as fp32 and the FMA units form
// the products, with a barrier in place of a launch: 64 x 32 takes 12 us with the host's part, 92 there.
//
// A thread adds up 2 x 2 elements of a product, both operands four steps of k at a time: rows of X by
// rows of X (A = X X^T, and A A, since A is symmetric), or rows of B by columns of X.  Where a square
// product has fewer such tiles than the CTA has threads, neighbouring lanes share out k and add up
// by shuffles.  Rows are padded with zeros to multiples of four, and by four more where their
// stride would be an even number of 16-byte units: 16-byte reads of eight rows then meet no bank twice.
#include <atomic>

#include "common.cuh"
#include "ns.hpp"

namespace fsdp {
namespace {

constexpr int kTinyThreads = 512;
constexpr int64_t kTinySide = 64;
constexpr int64_t kTinySmem = 200 * 1024;
// m^2 (2 n + m), a step's multiplications: above, one SM's FMA units take longer than the tiles
// of the products' kernels (64 x 128: 60 us against 92; 64 x 256: 110).
constexpr int64_t kTinyWork = 1200000;

struct TinySteps {
    float f[kNsMaxSteps][3];
    int32_t steps;
};

__host__ __device__ inline int pad4(int n) { return (n + 3) / 4 * 4; }
__host__ __device__ inline int tiny_ld(int n) { return (pad4(n) / 4) % 2 ? pad4(n) : pad4(n) + 4; }

__device__ __forceinline__ float tiny_get(const void* p, int64_t i, int bf16) {
    return bf16 ? bf16f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    s = __fmaf_rn(a.x, b.x, s);
    s = __fmaf_rn(a.y, b.y, s);
    s = __fmaf_rn(a.z, b.z, s);
    return __fmaf_rn(a.w, b.w, s);
}

// f(i, j, sum over k of r[i][k] r[j][k]) for all i, j below mp, in 2 x 2 tiles.
template <class F>
__device__ __forceinline__ void tiny_gram(const float* r, int ld, int mp, int kp, int tid, F&& f) {
    const int side = mp / 2, tiles = side * side;
    int slices = 1;                              // lanes that share a tile's k
    while (slices < 32 && 2 * slices * tiles <= kTinyThreads) slices *= 2;
    const int slice = tid % slices;
    for (int base = 0; base < tiles; base += kTinyThreads / slices) {
        const int tile = base + tid / slices;
        const bool have = tile < tiles;
        const int i = have ? tile / side * 2 : 0, j = have ? tile % side * 2 : 0;
        const float *const a = r + i * ld, *const b = r + j * ld;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 4 * slice; have && k < kp; k += 4 * slices) {
            const float4 a0 = ld4(a + k), a1 = ld4(a + ld + k), b0 = ld4(b + k), b1 = ld4(b + ld + k);
            s[0] = dot4(a0, b0, s[0]);
            s[1] = dot4(a0, b1, s[1]);
            s[2] = dot4(a1, b0, s[2]);
            s[3] = dot4(a1, b1, s[3]);
        }
        for (int o = 1; o < slices; o *= 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
        if (have && slice == 0) {
            f(i, j, s[0]);
            f(i, j + 1, s[1]);
            f(i + 1, j, s[2]);
            f(i + 1, j + 1, s[3]);
        }
    }
}

__global__ void __launch_bounds__(kTinyThreads)
k_ns_tiny(const __grid_constant__ NsMatrices src, const __grid_constant__ NsMatrices dst, int m, int n, float eps,
          const __grid_constant__ TinySteps st) {
    extern __shared__ __align__(16) float tiny_smem[];
    __shared__ double part[kTinyThreads / 32];
    const int tid = threadIdx.x, mat = blockIdx.x;
    const int mp = pad4(m), np = pad4(n), ldx = tiny_ld(n), lda = tiny_ld(m);
    float *x = tiny_smem, *y = x + mp * ldx, *const a = y + mp * ldx, *const b = a + mp * lda;
    for (int i = tid; i < 2 * mp * (ldx + lda); i += kTinyThreads) tiny_smem[i] = 0.f;
    __syncthreads();
    pdl_wait();
    // the matrix, whichever of its sides is the longer one along x's rows, and its sum of squares
    const bool tall = src.tall >> mat & 1;
    const int rows = tall ? n : m, cols = tall ? m : n;
    double square = 0.0;
    for (int i = tid; i < rows * cols; i += kTinyThreads) {
        const int r = i / cols, c = i - r * cols;
        const float v = tiny_get(src.p[mat], r * src.ld[mat] + c, src.bf16);
        x[tall ? c * ldx + r : r * ldx + c] = v;
        square += double(__fmul_rn(v, v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) square += __shfl_xor_sync(0xffffffffu, square, o);
    if ((tid & 31) == 0) part[tid >> 5] = square;
    __syncthreads();
    square = 0.0;
    for (int k = 0; k < kTinyThreads / 32; ++k) square += part[k];
    const double norm = sqrt(square);
    const float factor = float(1.0 / (norm < double(eps) ? double(eps) : norm));         // a NaN stays
    for (int i = tid; i < m * n; i += kTinyThreads) x[i / n * ldx + i % n] *= factor;
    __syncthreads();
    for (int k = 0; k < st.steps; ++k) {
        const float fa = st.f[k][0], fb = st.f[k][1], fc = st.f[k][2];
        tiny_gram(x, ldx, mp, np, tid, [&](int i, int j, float v) { a[i * lda + j] = v; });
        __syncthreads();
        tiny_gram(a, lda, mp, mp, tid, [&](int i, int j, float v) { b[i * lda + j] = __fmaf_rn(fc, v, __fmul_rn(fb, a[i * lda + j])); });
        __syncthreads();
        // X' = a X + B X, 2 x 2 elements a thread
        const int wide = np / 2;
        for (int t = tid; t < mp / 2 * wide; t += kTinyThreads) {
            const int i = t / wide * 2, j = t % wide * 2;
            const float *const b0 = b + i * lda, *const b1 = b0 + lda;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int l = 0; l < mp; l += 4) {
                const float4 p = ld4(b0 + l), q = ld4(b1 + l);
                const float pp[4] = {p.x, p.y, p.z, p.w}, qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = *reinterpret_cast<const float2*>(x + (l + e) * ldx + j);
                    s[0] = __fmaf_rn(pp[e], v.x, s[0]);
                    s[1] = __fmaf_rn(pp[e], v.y, s[1]);
                    s[2] = __fmaf_rn(qq[e], v.x, s[2]);
                    s[3] = __fmaf_rn(qq[e], v.y, s[3]);
                }
            }
            const float2 u = *reinterpret_cast<const float2*>(x + i * ldx + j), v = *reinterpret_cast<const float2*>(x + (i + 1) * ldx + j);
            *reinterpret_cast<float2*>(y + i * ldx + j) = make_float2(__fmaf_rn(fa, u.x, s[0]), __fmaf_rn(fa, u.y, s[1]));
            *reinterpret_cast<float2*>(y + (i + 1) * ldx + j) = make_float2(__fmaf_rn(fa, v.x, s[2]), __fmaf_rn(fa, v.y, s[3]));
        }
        __syncthreads();
        float* const z = x;
        x = y;
        y = z;
    }
    for (int i = tid; i < rows * cols; i += kTinyThreads) {
        const int r = i / cols, c = i - r * cols;
        const float v = x[tall ? c * ldx + r : r * ldx + c];
        const int64_t at = r * dst.ld[mat] + c;
        if (dst.bf16) static_cast<uint16_t*>(dst.p[mat])[at] = to_bf16(v);
        else static_cast<float*>(dst.p[mat])[at] = v;
    }
}

size_t tiny_bytes(int64_t m, int64_t n) { return size_t(2 * pad4(int(m)) * (tiny_ld(int(n)) + tiny_ld(int(m)))) * 4; }

}  // namespace

bool use_ns_tiny(int64_t m, int64_t n) {
    return m <= kTinySide && n <= (int64_t(1) << 20) && m * m * (2 * n + m) <= kTinyWork && tiny_bytes(m, n) <= size_t(kTinySmem);
}

cudaError_t launch_ns_tiny(const NsMatrices& src, const NsMatrices& dst, int batch, int64_t m, int64_t n, float eps, const float* coeffs,
                           int steps, const float* usual, cudaStream_t st) {
    TinySteps s = {};
    s.steps = steps;
    for (int k = 0; k < steps; ++k)
        for (int i = 0; i < 3; ++i) s.f[k][i] = coeffs ? coeffs[3 * k + i] : usual[i];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    static std::atomic<uint64_t> prepared{0};
    if (e == cudaSuccess && (dev >= 64 || !(prepared.load(std::memory_order_relaxed) >> dev & 1))) {
        e = cudaFuncSetAttribute(k_ns_tiny, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTinySmem));
        if (e == cudaSuccess && dev < 64) prepared.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return e;
    return launch(k_ns_tiny, dim3(unsigned(batch)), dim3(kTinyThreads), tiny_bytes(m, n), st, src, dst, int(m), int(n), eps, s);
}

}  // namespace fsdp
