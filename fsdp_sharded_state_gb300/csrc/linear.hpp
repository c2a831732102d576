// linear.hpp -- host-side types and launchers of the linear-layer kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "philox.cuh"

namespace fsdp {

// A linear layer's three products: out[r][c] = sum over k of R[r, k] C[c, k].
//   forward   R = x,    C = w,    K = in features
//   dgrad     R = dz,   C = w^T,  K = out features
//   wgrad     R = dz^T, C = x^T,  K = rows of the batch
enum LinMode { kForward = 0, kDgrad = 1, kWgrad = 2 };

// The epilogue of a product; pointers in the output's element type.
struct LinEpi {
    void* out;
    int64_t ldo;
    const void* bias;          // forward
    const void* residual;      // forward, dgrad: added last
    int64_t ldr;
    void* preact;              // forward: written; dgrad: read
    int64_t ldz;
    int64_t rows, cols;        // of out
    int32_t act;               // fsdp_act
    int32_t accumulate;        // wgrad: out += instead of out =
    int32_t vec;               // every matrix here has rows aligned to 16 bytes (1), 32 bytes (2), or not (0)
    void* db;                  // wgrad: the column sums of dz, or NULL
    const void* dz;            // and dz itself (fp32: as the caller holds it)
    int64_t lddz, dz_rows;
    int32_t dz_vec;            // 16-byte aligned rows
    Drop drop;
};

// One operand as the tensor maps see it: `planes` row-major bf16 matrices of rows x cols,
// 16-byte aligned base, ld a multiple of 8 elements, plane a multiple of 8 elements.
struct LinOperand {
    const void* ptr;
    int64_t rows, cols, ld, plane;
};

struct LinProblem {
    LinMode mode;
    int64_t K;
    LinOperand rows_op, cols_op;   // R and C, as the caller stores them
    int planes;                // 1: bf16 operands; 3: fp32 operands as three bf16 terms
    bool out_bf16;
    LinEpi epi;
    int slabs;                 // wgrad: K ranges that may get partial sums of their own (0: none), and
    float* partial;            // room for them, wgrad_slab_floats() floats
};

// wgrad with a small out: how many slabs its rows are cut into, a cluster of kSlabSplits CTAs on
// each tile of each (0: out alone fills the device), and the floats of their partial sums
// (out's rows padded to 8 columns, then db).
constexpr int kSlabSplits = 4;
int wgrad_slabs(int64_t rows, int64_t in, int64_t out);
int64_t wgrad_slab_floats(int64_t rows, int64_t in, int64_t out);
cudaError_t launch_wgrad_slabs(const LinProblem& p, cudaStream_t st);
// The sum of `parts` partial sums of out ([parts][rows][ld]) and db ([parts][rows]), in order, into ep's.
cudaError_t launch_join(const float* part, const float* db_part, int parts, int64_t rows, int64_t cols, int64_t ld, const LinEpi& ep,
                        bool out_bf16, cudaStream_t st);

cudaError_t launch_linear_forward(const LinProblem& p, cudaStream_t st);
cudaError_t launch_linear_dgrad(const LinProblem& p, cudaStream_t st);
cudaError_t launch_linear_wgrad(const LinProblem& p, cudaStream_t st);
// The CTA-pair kernels with bf16 operands and results, tiles of 256 x bn.
cudaError_t launch_pair_forward(const LinProblem& p, int bn, cudaStream_t st);
cudaError_t launch_pair_dgrad(const LinProblem& p, int bn, cudaStream_t st);

// forward (x: its x) or dgrad (x: dz) of a few rows, operands as the caller stores them.
struct SkinnyProblem {
    LinMode mode;
    bool bf16;
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw, K;
    LinEpi epi;
};
cudaError_t launch_skinny(const SkinnyProblem& p, cudaStream_t st);
bool use_skinny(LinMode mode, bool bf16, int64_t rows, int64_t in, int64_t out);

// A small product of fp32 operands as the caller stores them: a x or dz, b w or (wgrad) x.
struct SmallProblem {
    LinMode mode;
    const float* a;
    int64_t lda;
    const float* b;
    int64_t ldb, K;
    bool out_bf16;             // wgrad
    float* partial;            // wgrad: small_slab_floats() floats
    LinEpi epi;
};
cudaError_t launch_small(const SmallProblem& p, cudaStream_t st);
bool use_small(LinMode mode, int64_t rows, int64_t in, int64_t out);
int64_t small_slab_floats(int64_t rows, int64_t in, int64_t out);

// Operands brought into the form of LinOperand: a bf16 matrix copied to aligned rows, or
// an fp32 matrix split into three bf16 planes (see linear_pack.cu).  Up to two per launch.
struct PackJob {
    const void* src;
    int64_t rows, cols, ld;
    void* dst;
    int64_t dld, plane;
};
cudaError_t launch_pack(const PackJob* jobs, int n, bool f32, cudaStream_t st);

// y = residual + drop(x); drop.on = 0 copies.
cudaError_t launch_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy, bool bf16,
                           int64_t rows, int64_t cols, const Drop& d, cudaStream_t st);

// Read and clear the wait words of the linear kernels (synchronous), one per translation unit.
cudaError_t take_wait_error_forward(unsigned int* flag);
cudaError_t take_wait_error_forward_pair(unsigned int* flag);
cudaError_t take_wait_error_dgrad(unsigned int* flag);
cudaError_t take_wait_error_dgrad_pair(unsigned int* flag);
cudaError_t take_wait_error_wgrad(unsigned int* flag);

}  // namespace fsdp
