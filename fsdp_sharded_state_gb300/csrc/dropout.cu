// dropout.cu -- y = residual + drop(x) over a row-major matrix, the mask drawn where it is
// used (philox.cuh) and never stored; backward is the same call on the gradient.
#include "common.cuh"
#include "linear.hpp"

namespace fsdp {
namespace {

constexpr int kDropThreads = 256;

__device__ __forceinline__ float get(const uint16_t* p) { return bf16f(*p); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// A thread: 4 columns of one row, one generator block.
template <typename T>
__global__ void __launch_bounds__(kDropThreads)
k_dropout(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy, int64_t rows, int64_t cols, int64_t quads,
          const Drop d) {
    pdl_wait();
    const int64_t i = int64_t(blockIdx.x) * kDropThreads + threadIdx.x;
    const int64_t r = i / quads, q = i - r * quads;
    if (r >= rows) return;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (d.on) w = drop_words(d, r, q);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t c = q * 4 + k;
        if (c >= cols) break;
        float v = get(x + r * ldx + c);
        if (d.on) v = drop1(d, ws[k], v);
        if (res) v += get(res + r * ldr + c);
        put(y + r * ldy + c, v);
    }
}

template <typename T>
cudaError_t run(const void* x, int64_t ldx, const void* res, int64_t ldr, void* y, int64_t ldy, int64_t rows, int64_t cols,
                const Drop& d, cudaStream_t st) {
    const int64_t quads = (cols + 3) / 4, blocks = (rows * quads + kDropThreads - 1) / kDropThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch(k_dropout<T>, dim3(unsigned(blocks)), dim3(kDropThreads), 0, st, static_cast<const T*>(x), ldx,
                  static_cast<const T*>(res), ldr, static_cast<T*>(y), ldy, rows, cols, quads, d);
}

}  // namespace

cudaError_t launch_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy, bool bf16,
                           int64_t rows, int64_t cols, const Drop& d, cudaStream_t st) {
    return bf16 ? run<uint16_t>(x, ldx, residual, ldr, y, ldy, rows, cols, d, st)
                : run<float>(x, ldx, residual, ldr, y, ldy, rows, cols, d, st);
}

}  // namespace fsdp
