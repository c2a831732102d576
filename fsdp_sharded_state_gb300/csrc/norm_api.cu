// norm_api.cu -- the extern "C" entry points of layer norm: argument checks and launches.
// Every check runs before the first launch.
#include <cmath>

#include "internal.hpp"
#include "norm.hpp"

using namespace fsdp;
using namespace fsdp::detail;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxElems = int64_t(1) << 40;

bool known(int32_t dtype) { return dtype == FSDP_F32 || dtype == FSDP_BF16; }

int check_dims(int64_t rows, int64_t cols, int32_t dtype) {
    if (!known(dtype)) return FSDP_EDTYPE;
    if (rows < 0 || cols < 1) return FSDP_ESHAPE;
    if (rows > kMaxRows || cols > kNormMaxCols || rows * cols > kMaxElems) return FSDP_EOVERFLOW;
    return FSDP_OK;
}

int check_matrix(const void* p, int64_t cols, int64_t ld, int es) {
    if (!p) return FSDP_EINVAL;
    if (reinterpret_cast<uintptr_t>(p) % unsigned(es)) return FSDP_EALIGN;
    if (ld < cols) return FSDP_ESHAPE;
    if (ld > kMaxRows) return FSDP_EOVERFLOW;
    return FSDP_OK;
}

int check_vector(const void* p, int es) { return reinterpret_cast<uintptr_t>(p) % unsigned(es) ? FSDP_EALIGN : FSDP_OK; }

// Whether a matrix's rows are whole chunks of 16 bytes.
bool rows16(const void* p, int64_t cols, int64_t ld, int es) { return !p || (aligned16(p) && ld * es % 16 == 0 && cols * es % 16 == 0); }

}  // namespace

extern "C" {

int fsdp_layernorm_forward(int64_t rows, int64_t cols, int32_t elem_dtype, const void* x, int64_t ldx, const void* weight,
                           const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd, fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_layernorm_forward");
    int rc = check_dims(rows, cols, elem_dtype);
    if (rc) return rc;
    const int es = elem_dtype == FSDP_F32 ? 4 : 2;
    if (!(eps > 0.f) || !std::isfinite(eps)) return FSDP_EINVAL;
    if (rows > 0 && ((rc = check_matrix(x, cols, ldx, es)) || (rc = check_matrix(y, cols, ldy, es)))) return rc;
    if ((rc = check_vector(weight, es)) || (rc = check_vector(bias, es)) || (rc = check_vector(mean, 4)) || (rc = check_vector(rstd, 4)))
        return rc;
    if (rows == 0) return FSDP_OK;
    NormProblem p = {};
    p.rows = rows;
    p.cols = cols;
    p.bf16 = elem_dtype == FSDP_BF16;
    p.vec = rows16(x, cols, ldx, es) && rows16(y, cols, ldy, es);
    p.x = x;
    p.ldx = ldx;
    p.weight = weight;
    p.bias = bias;
    p.eps = eps;
    p.y = y;
    p.ldy = ldy;
    p.mean = mean;
    p.rstd = rstd;
    const cudaError_t e = launch_norm_forward(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "k_norm_forward launch");
}

size_t fsdp_layernorm_workspace_bytes(int64_t rows, int64_t cols) {
    return check_dims(rows, cols, FSDP_F32) ? 0 : size_t(norm_partial_floats(rows, cols)) * 4;
}

int fsdp_layernorm_backward(int64_t rows, int64_t cols, int32_t elem_dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                            const float* mean, const float* rstd, const void* weight, const void* residual, int64_t ldr, void* dx,
                            int64_t lddx, void* dw, void* db, int32_t grad_dtype, int32_t accumulate, void* workspace,
                            size_t workspace_bytes, fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_layernorm_backward");
    int rc = check_dims(rows, cols, elem_dtype);
    if (rc) return rc;
    if (!known(grad_dtype)) return FSDP_EDTYPE;
    const int es = elem_dtype == FSDP_F32 ? 4 : 2, gs = grad_dtype == FSDP_F32 ? 4 : 2;
    if (rows > 0) {
        if ((rc = check_matrix(dy, cols, lddy, es)) || (rc = check_matrix(x, cols, ldx, es)) || (rc = check_matrix(dx, cols, lddx, es)))
            return rc;
        if (!mean || !rstd) return FSDP_EINVAL;
        if (residual && (rc = check_matrix(residual, cols, ldr, es))) return rc;
    }
    if ((rc = check_vector(mean, 4)) || (rc = check_vector(rstd, 4)) || (rc = check_vector(weight, es)) || (rc = check_vector(dw, gs)) ||
        (rc = check_vector(db, gs)))
        return rc;
    if (workspace && !aligned16(workspace)) return FSDP_EALIGN;
    if ((dw || db) && rows > 0 && (!workspace || workspace_bytes < fsdp_layernorm_workspace_bytes(rows, cols))) return FSDP_EINVAL;
    NormProblem p = {};
    p.rows = rows;
    p.cols = cols;
    p.bf16 = elem_dtype == FSDP_BF16;
    p.vec = rows16(x, cols, ldx, es) && rows16(dy, cols, lddy, es) && rows16(dx, cols, lddx, es) && rows16(residual, cols, ldr, es);
    p.x = x;
    p.ldx = ldx;
    p.weight = weight;
    p.y = dx;
    p.ldy = lddx;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.dy = dy;
    p.lddy = lddy;
    p.residual = residual;
    p.ldr = ldr;
    p.dw = dw;
    p.db = db;
    p.grad_bf16 = grad_dtype == FSDP_BF16;
    p.accumulate = accumulate != 0;
    p.partial = static_cast<float*>(workspace);
    const cudaError_t e = launch_norm_backward(p, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "k_norm_backward launch");
}

}  // extern "C"
