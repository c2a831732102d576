// ns_prep.cu -- what comes before the products of Newton-Schulz steps: the sum of squares of
// each matrix, and the first X as two fp16 terms.
//
// Both are bound by HBM (the matrix read twice, 4 bytes an element written).  Squares are added in
// fp32, a thread's sum of many with what each addition rounds carried along, in a fixed order: an
// error of the norm scales all of X alike.  (There are two fp64 units an SM: sums, root and quotient
// in 64 bits took longer than the reads.)
#include <cuda_fp16.h>

#include "common.cuh"
#include "ns.hpp"

namespace fsdp {
namespace {

constexpr int kPrepThreads = 256;

__device__ __forceinline__ float ns_get(const void* p, int64_t i, int bf16) {
    return bf16 ? bf16f(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// The sum over a CTA's threads, in thread 0.
__device__ __forceinline__ float block_sum(float v) {
    __shared__ float part[kPrepThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.f;
        for (int k = 0; k < kPrepThreads / 32; ++k) v += part[k];
    }
    return v;
}

// The source's elements in the order of its rows, kStrip at a time; block (part, matrix).
constexpr int kStrip = 16 * kPrepThreads;

__global__ void __launch_bounds__(kPrepThreads)
k_ns_squares(const __grid_constant__ NsMatrices src, int64_t rows, int64_t cols, float* partial) {
    pdl_wait();
    pdl_trigger();
    const int mat = blockIdx.y;
    const bool tall = src.tall >> mat & 1;
    const int64_t R = tall ? cols : rows, W = tall ? rows : cols;    // the source's own rows and width
    const int64_t ld = src.ld[mat], n = R * W;
    const void* const p = src.p[mat];
    float total = 0.f, lost = 0.f;
    for (int64_t base = int64_t(blockIdx.x) * kStrip; base < n; base += int64_t(gridDim.x) * kStrip) {
        int64_t i = base + threadIdx.x;
        int64_t r = i / W, c = i - r * W;
        float v[16], s = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            v[k] = i < n ? ns_get(p, r * ld + c, src.bf16) : 0.f;
            i += kPrepThreads;
            c += kPrepThreads;
            while (c >= W) {
                c -= W;
                ++r;
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) s = __fmaf_rn(v[k], v[k], s);
        add_carefully(s, total, lost);
    }
    total = block_sum(total);
    if (threadIdx.x == 0) partial[mat * gridDim.x + blockIdx.x] = total;
}

// A tile of 64 x 64 of the planes goes through shared memory, so that reads follow the source's
// rows in either orientation and writes the planes'.
__global__ void __launch_bounds__(kPrepThreads)
k_ns_pack(const __grid_constant__ NsMatrices src, const NsPlanes out, const float* partial, int parts, float scale, float eps,
          int tiles_n) {
    __shared__ float tile[64][65];
    __shared__ float factor;
    pdl_wait();
    pdl_trigger();
    const int mat = blockIdx.y, tid = threadIdx.x;
    const bool tall = src.tall >> mat & 1;
    const int64_t m0 = int64_t(blockIdx.x / tiles_n) * 64, n0 = int64_t(blockIdx.x % tiles_n) * 64, ld = src.ld[mat];
    const int64_t r0 = tall ? n0 : m0, c0 = tall ? m0 : n0;          // the source's tile
    const int64_t R = tall ? out.cols : out.rows, W = tall ? out.rows : out.cols;
    const float* const p32 = static_cast<const float*>(src.p[mat]) + r0 * ld + c0;
    // the tile's loads go out before the norm is there: 4 x 4 elements a thread
    const bool vec = !src.bf16 && ((reinterpret_cast<uintptr_t>(p32) | uintptr_t(ld * 4)) & 15) == 0 && r0 + 64 <= R && c0 + 64 <= W;
    float v[16];
    if (vec) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 q = ld4(p32 + ((tid >> 4) + 16 * k) * ld + (tid & 15) * 4);
            v[4 * k] = q.x; v[4 * k + 1] = q.y; v[4 * k + 2] = q.z; v[4 * k + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int64_t r = r0 + (tid >> 6) + 4 * k, c = c0 + (tid & 63);
            v[k] = r < R && c < W ? ns_get(src.p[mat], r * ld + c, src.bf16) : 0.f;
        }
    }
    float square = 0.f;
    for (int k = tid; k < parts; k += kPrepThreads) square += partial[mat * parts + k];
    square = block_sum(square);
    if (tid == 0) {
        const float norm = sqrtf(square);
        factor = scale / (norm < eps ? eps : norm);              // a NaN stays
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int y = vec ? (tid >> 4) + 16 * (k / 4) : (tid >> 6) + 4 * k, x = vec ? (tid & 15) * 4 + k % 4 : tid & 63;
        if (tall) tile[x][y] = v[k];
        else tile[y][x] = v[k];
    }
    __syncthreads();
    uint16_t* const dst = out.p + 2 * int64_t(mat) * out.plane;
    const float f = factor;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int row = (tid >> 3) + 32 * k, col = (tid & 7) * 8;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = tile[row][col + 2 * j] * f, b = tile[row][col + 2 * j + 1] * f;
            const __half2 h = __floats2half2_rn(a, b);
            const float2 g = __half22float2(h);
            const __half2 l = __floats2half2_rn(a - g.x, b - g.y);
            hi[j] = *reinterpret_cast<const uint32_t*>(&h);
            lo[j] = *reinterpret_cast<const uint32_t*>(&l);
        }
        // the planes are padded to whole tiles
        uint16_t* const q = dst + (m0 + row) * out.ld + n0 + col;
        stu4(q, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        stu4(q + out.plane, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
}

}  // namespace

int ns_parts(int64_t numel) {
    const int64_t n = (numel + kStrip - 1) / kStrip;
    return int(n < 1 ? 1 : n < kNsMaxParts ? n : kNsMaxParts);
}

cudaError_t launch_ns_squares(const NsMatrices& src, int batch, int64_t rows, int64_t cols, float* partial, int parts, cudaStream_t st) {
    return launch(k_ns_squares, dim3(unsigned(parts), unsigned(batch)), dim3(kPrepThreads), 0, st, src, rows, cols, partial);
}

cudaError_t launch_ns_pack(const NsMatrices& src, int batch, const NsPlanes& out, const float* partial, int parts, float scale, float eps,
                           cudaStream_t st) {
    const int64_t tm = (out.rows + 63) / 64, tn = (out.cols + 63) / 64;
    if (tm * tn > INT32_MAX) return cudaErrorInvalidValue;
    return launch(k_ns_pack, dim3(unsigned(tm * tn), unsigned(batch)), dim3(kPrepThreads), 0, st, src, out, partial, parts, scale, eps,
                  int(tn));
}

}  // namespace fsdp
