// norm.hpp -- host-side types and launchers of the layer-norm kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fsdp {

// Rows of up to kNormMaxCols columns are held in registers from their load to their store.
constexpr int64_t kNormMaxCols = 65536;

// Matrices and vectors in the call's element type; weight, bias, residual, mean, rstd, dw and
// db may be NULL (mean and rstd only in forward).
struct NormProblem {
    int64_t rows, cols;
    bool bf16;
    bool vec;                       // every matrix has rows of whole 16-byte chunks
    const void* x;
    int64_t ldx;
    const void* weight;
    const void* bias;
    void* y;                        // forward: y; backward: dx
    int64_t ldy;
    float* mean;
    float* rstd;
    float eps;
    const void* dy;                 // backward
    int64_t lddy;
    const void* residual;
    int64_t ldr;
    void* dw;
    void* db;
    bool grad_bf16, accumulate;
    float* partial;                 // norm_partial_floats()
};

// Floats of backward's partial sums of dw and db.
int64_t norm_partial_floats(int64_t rows, int64_t cols);

cudaError_t launch_norm_forward(const NormProblem& p, cudaStream_t st);
cudaError_t launch_norm_backward(const NormProblem& p, cudaStream_t st);
cudaError_t take_wait_error_norm_forward(unsigned int* flag);
cudaError_t take_wait_error_norm_backward(unsigned int* flag);

}  // namespace fsdp
