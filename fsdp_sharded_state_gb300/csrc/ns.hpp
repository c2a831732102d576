// ns.hpp -- host-side types and launchers of the Newton-Schulz kernels.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace fsdp {

constexpr int kNsMaxBatch = 64;                 // matrices of a launch
constexpr int kNsMaxSteps = 64;
// The least eps: below it, squares that are lost below fp32's range could matter.
constexpr float kNsLeastEps = 1e-16f;

// A batch of fp32 matrices as two fp16 terms each: matrix i's high terms at p + 2 i plane, its
// low ones a plane on; rows of ld elements.  Buffers are padded to multiples of 256 rows and
// columns, so that whole tiles are stored without a bound; what lies past rows x cols is never
// read (the tensor map ends there).
struct NsPlanes {
    uint16_t* p;
    int64_t rows, cols, ld, plane;
};

// Where the last step's result goes, or where the first one's matrix comes from: matrix i is
// rows x cols of the planes, or (bit i of `tall`) its transpose.
struct NsMatrices {
    void* p[kNsMaxBatch];
    int64_t ld[kNsMaxBatch];
    uint64_t tall;
    int32_t bf16;
};

enum NsEpilogue { kNsGram = 0, kNsPoly = 1, kNsStep = 2, kNsLast = 3, kNsMul = 4 };

// One product of a step, over the whole batch.
//   gram   A = alpha X X^T                    x: X, out: A       (symmetric: half the tiles)
//   poly   B = alpha A A + beta A + diag I    x: A, out: B       (symmetric)
//   mul    alpha B A of two polynomials of one symmetric matrix: x, y, out (symmetric)
//   step   X' = alpha Q X                     x: Q, y: X, out: X'
//   last   the same, into `last`
struct NsProduct {
    int batch;
    NsPlanes x, y, out;
    float alpha, beta, diag;
    const NsMatrices* last;
};

cudaError_t launch_ns_gram(const NsProduct& p, cudaStream_t st);
cudaError_t launch_ns_poly(const NsProduct& p, cudaStream_t st);
cudaError_t launch_ns_mul(const NsProduct& p, cudaStream_t st);
cudaError_t launch_ns_step(const NsProduct& p, cudaStream_t st);
cudaError_t launch_ns_last(const NsProduct& p, cudaStream_t st);
cudaError_t take_wait_error_ns_gram(unsigned int* flag);
cudaError_t take_wait_error_ns_poly(unsigned int* flag);
cudaError_t take_wait_error_ns_mul(unsigned int* flag);
cudaError_t take_wait_error_ns_step(unsigned int* flag);
cudaError_t take_wait_error_ns_last(unsigned int* flag);

// Estimated times in us, from the sizes (x, y, batch) alone.
float cost_ns_gram(const NsProduct& p);
float cost_ns_mul(const NsProduct& p);
float cost_ns_step(const NsProduct& p);

// Blocks that sum a matrix's squares (a float each), at most kNsMaxParts.
constexpr int kNsMaxParts = 608;
int ns_parts(int64_t numel);
// partial[i][part] of the batch's source matrices (rows x cols, or transposed).
cudaError_t launch_ns_squares(const NsMatrices& src, int batch, int64_t rows, int64_t cols, float* partial, int parts, cudaStream_t st);
// The planes of scale / max(norm, eps) times the source, norm from the partial sums.
cudaError_t launch_ns_pack(const NsMatrices& src, int batch, const NsPlanes& out, const float* partial, int parts, float scale, float eps,
                           cudaStream_t st);

#ifdef __CUDACC__
// The next kernel of a run may start its set-up beside this one, which is small or about to end; it
// waits, as every kernel does, for this one's end before it touches memory.  Not before this
// one's own wait: then it would be there while the one before still runs.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// total += v, with what the addition rounds off kept in `lost` for the next.
__device__ __forceinline__ void add_carefully(float v, float& total, float& lost) {
    const float y = v - lost, t = total + y;
    lost = t - total - y;
    if (!(lost == lost)) lost = 0.f;             // an infinite total
    total = t;
}
#endif

// Small matrices: from the source to the result in one launch, without the workspace.
bool use_ns_tiny(int64_t m, int64_t n);
cudaError_t launch_ns_tiny(const NsMatrices& src, const NsMatrices& dst, int batch, int64_t m, int64_t n, float eps, const float* coeffs,
                           int steps, const float* usual, cudaStream_t st);

// Layout of the workspace of a batch (byte offsets); m and n are the shorter and the longer side,
// chunk the matrices that pass through it at once.
struct NsWork {
    int64_t m, n;
    int chunk;
    int64_t x0, x1, square[4], partial, end;
};
NsWork ns_work(int64_t rows, int64_t cols, int64_t count);
// Scales of a schedule of coefficients, [steps][3] (NULL: the default each step); false: a step may
// leave the range that the planes hold.
struct NsScales {
    float x[kNsMaxSteps + 1], a[kNsMaxSteps], b[kNsMaxSteps];    // of X, A and B of each step
    double top[kNsMaxSteps + 1], gain[kNsMaxSteps];              // bounds: of X's singular values, of B's eigenvalues
};
bool ns_scales(const float* coeffs, int steps, NsScales* s);
// From source matrices and their partial sums (which small ones do not need) to `dst`; one chunk.
// groups: steps may share a pass over X, at a cost in precision.
cudaError_t ns_run(const NsWork& w, unsigned char* ws, int batch, const NsMatrices& src, const NsMatrices& dst, int parts, float eps,
                   const float* coeffs, int steps, const NsScales& sc, bool groups, cudaStream_t st);

}  // namespace fsdp
