// linear_api.cu -- the extern "C" entry points of the layer operators (linear layers and
// dropout): argument checks, operand preparation and launches.  Every check runs before the
// first launch.
#include <algorithm>
#include <cmath>

#include "internal.hpp"
#include "linear.hpp"

using namespace fsdp;
using namespace fsdp::detail;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxElems = int64_t(1) << 40;              // of a matrix: sizes in bytes, three planes of it too, stay far below 2^63

int elem_size(int32_t dtype) { return dtype == FSDP_F32 ? 4 : 2; }
bool known(int32_t dtype) { return dtype == FSDP_F32 || dtype == FSDP_BF16; }

int check_dims(int64_t rows, int64_t in, int64_t out, int32_t dtype) {
    if (!known(dtype)) return FSDP_EDTYPE;
    if (rows < 0 || in < 1 || out < 1) return FSDP_ESHAPE;
    if (rows > kMaxDim || in > kMaxDim || out > kMaxDim) return FSDP_EOVERFLOW;
    if (rows * in > kMaxElems || rows * out > kMaxElems || in * out > kMaxElems) return FSDP_EOVERFLOW;
    return FSDP_OK;
}

// A matrix of rows x cols: present, aligned to its element, rows of at least cols elements.
int check_matrix(const void* p, int64_t cols, int64_t ld, int esize) {
    if (!p) return FSDP_EINVAL;
    if (reinterpret_cast<uintptr_t>(p) % unsigned(esize)) return FSDP_EALIGN;
    if (ld < cols) return FSDP_ESHAPE;
    if (ld > kMaxDim) return FSDP_EOVERFLOW;
    return FSDP_OK;
}

int check_vector(const void* p, int esize) {
    return p && reinterpret_cast<uintptr_t>(p) % unsigned(esize) ? FSDP_EALIGN : FSDP_OK;
}

int make_drop(const fsdp_dropout_spec* s, int64_t rows, Drop* d) {
    *d = Drop{};
    if (!s) return FSDP_OK;
    if (!(s->p >= 0.0) || !(s->p < 1.0) || s->row0 < 0) return FSDP_EINVAL;
    if (s->row0 > INT64_MAX - rows) return FSDP_EOVERFLOW;
    d->thr = uint32_t(std::floor(s->p * 4294967296.0));
    d->on = s->p > 0.0;
    d->scale = float(1.0 / (1.0 - s->p));
    for (uint32_t i = 0; i < 10; ++i) {
        d->key[i][0] = uint32_t(s->seed) + i * 0x9E3779B9u;
        d->key[i][1] = uint32_t(s->seed >> 32) + i * 0xBB67AE85u;
    }
    d->layer = s->layer;
    d->row0 = s->row0;
    return FSDP_OK;
}

bool rows16(const void* p, int64_t ld, int esize) { return aligned16(p) && ld * esize % 16 == 0; }

// How the rows of an epilogue's matrix are aligned: to 32 bytes (2), 16 (1), or not (0); a
// matrix that is not there is aligned.
int row_class(const void* p, int64_t ld, int esize) {
    if (!p) return 2;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * esize);
    return a % 32 == 0 ? 2 : a % 16 == 0 ? 1 : 0;
}

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Elements of a packed row (whole lines of 128 bytes, so that a box row of 64 elements is one
// line: with rows of 16-byte multiples, each is two, and 4000 x 4001 x 4001 took 120 us instead
// of 91), of one packed plane, and bytes of a packed operand.
int64_t packed_ld(int64_t cols) { return round_up(cols, 64); }
int64_t plane_elems(int64_t rows, int64_t cols) { return rows * packed_ld(cols); }
int64_t packed_bytes(int64_t rows, int64_t cols, int planes) { return round_up(planes * plane_elems(rows, cols) * 2, 256); }

// The operands of a product: a matrix that the tensor maps can read where it is, or its
// packed copy in the workspace.  The calls of a few rows (use_skinny) take no room for the
// weight, which they read where it is; the rows' own, a few KB, is taken whatever kernel runs.
struct Packer {
    unsigned char* ws;
    size_t left;
    PackJob jobs[2];
    int n = 0;

    int operand(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, LinOperand* o) {
        if (dtype == FSDP_BF16 && rows16(p, ld, 2)) {
            *o = LinOperand{p, rows, cols, ld, rows * ld};
            return FSDP_OK;
        }
        const int planes = dtype == FSDP_F32 ? 3 : 1;
        const int64_t need = packed_bytes(rows, cols, planes);
        if (!ws || left < size_t(need)) return FSDP_EINVAL;
        const int64_t dld = packed_ld(cols), plane = plane_elems(rows, cols);
        jobs[n++] = PackJob{p, rows, cols, ld, ws, dld, plane};
        *o = LinOperand{ws, rows, cols, dld, plane};
        ws += need;
        left -= size_t(need);
        return FSDP_OK;
    }
};

int run_product(LinProblem& p, Packer& pk, int32_t elem_dtype, cudaStream_t st) {
    cudaError_t e = launch_pack(pk.jobs, pk.n, elem_dtype == FSDP_F32, st);
    if (e != cudaSuccess) return cuda_fail(e, "k_pack launch");
    e = p.mode == kForward ? launch_linear_forward(p, st) : p.mode == kDgrad ? launch_linear_dgrad(p, st) : launch_linear_wgrad(p, st);
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "k_linear launch");
}

int run_small(LinMode mode, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t K, bool out_bf16, float* partial,
              const LinEpi& ep, cudaStream_t st) {
    const cudaError_t e = launch_small(
        SmallProblem{mode, static_cast<const float*>(a), lda, static_cast<const float*>(b), ldb, K, out_bf16, partial, ep}, st);
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "k_small launch");
}

int run_skinny(LinMode mode, int32_t dtype, const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t K, const LinEpi& ep,
               cudaStream_t st) {
    const cudaError_t e = launch_skinny(SkinnyProblem{mode, dtype == FSDP_BF16, x, ldx, w, ldw, K, ep}, st);
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "k_skinny launch");
}

// Floats of wgrad's partial sums.
int64_t partial_floats(int64_t rows, int64_t in, int64_t out, int32_t elem_dtype) {
    return std::max(wgrad_slab_floats(rows, in, out), elem_dtype == FSDP_F32 ? small_slab_floats(rows, in, out) : 0);
}

}  // namespace

extern "C" {

size_t fsdp_linear_workspace_bytes(int64_t rows, int64_t in, int64_t out, int32_t elem_dtype, int32_t aligned) {
    if (check_dims(rows, in, out, elem_dtype)) return 0;
    const size_t slabs = size_t(round_up(partial_floats(rows, in, out, elem_dtype) * 4, 256));
    if (elem_dtype == FSDP_BF16 && aligned) return slabs;
    const int planes = elem_dtype == FSDP_F32 ? 3 : 1;
    const int64_t x = packed_bytes(rows, in, planes), w = packed_bytes(out, in, planes), z = packed_bytes(rows, out, planes);
    auto weight = [&](LinMode mode) { return use_skinny(mode, elem_dtype == FSDP_BF16, rows, in, out) ? 0 : w; };
    return size_t(std::max({x + weight(kForward), z + weight(kDgrad), x + z})) + slabs;
}

int fsdp_linear_forward(int64_t rows, int64_t in, int64_t out, int32_t elem_dtype, const void* x, int64_t ldx, const void* w,
                        int64_t ldw, const void* bias, int32_t act, const fsdp_dropout_spec* drop, const void* residual,
                        int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldz, void* workspace, size_t workspace_bytes,
                        fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_linear_forward");
    int rc = check_dims(rows, in, out, elem_dtype);
    if (rc) return rc;
    const int es = elem_size(elem_dtype);
    if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU) return FSDP_EINVAL;
    if (rows > 0 && ((rc = check_matrix(x, in, ldx, es)) || (rc = check_matrix(y, out, ldy, es)))) return rc;
    if ((rc = check_matrix(w, in, ldw, es)) || (rc = check_vector(bias, es))) return rc;
    if (residual && (rc = check_matrix(residual, out, ldr, es))) return rc;
    if (preact && (rc = check_matrix(preact, out, ldz, es))) return rc;
    if (workspace && !aligned16(workspace)) return FSDP_EALIGN;
    LinProblem p = {};
    if ((rc = make_drop(drop, rows, &p.epi.drop))) return rc;
    if (rows == 0) return FSDP_OK;
    p.mode = kForward;
    p.K = in;
    p.planes = elem_dtype == FSDP_F32 ? 3 : 1;
    p.out_bf16 = elem_dtype == FSDP_BF16;
    LinEpi& ep = p.epi;
    ep.out = y;
    ep.ldo = ldy;
    ep.bias = bias;
    ep.residual = residual;
    ep.ldr = ldr;
    ep.preact = preact;
    ep.ldz = ldz;
    ep.rows = rows;
    ep.cols = out;
    ep.act = act;
    ep.vec = std::min({row_class(y, ldy, es), row_class(residual, ldr, es), row_class(preact, ldz, es)});
    if (bias && !aligned16(bias)) ep.vec = 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Packer pk{static_cast<unsigned char*>(workspace), workspace_bytes, {}};
    const bool skinny = use_skinny(kForward, elem_dtype == FSDP_BF16, rows, in, out);
    if (!skinny && (rc = pk.operand(w, out, in, ldw, elem_dtype, &p.cols_op))) return rc;
    if ((rc = pk.operand(x, rows, in, ldx, elem_dtype, &p.rows_op))) return rc;
    if (skinny) return run_skinny(kForward, elem_dtype, x, ldx, w, ldw, in, ep, st);
    if (elem_dtype == FSDP_F32 && use_small(kForward, rows, in, out))
        return run_small(kForward, x, ldx, w, ldw, in, false, nullptr, ep, st);
    return run_product(p, pk, elem_dtype, st);
}

int fsdp_linear_dgrad(int64_t rows, int64_t in, int64_t out, int32_t elem_dtype, const void* dz, int64_t lddz, const void* w,
                      int64_t ldw, int32_t act, const void* preact, int64_t ldz, const fsdp_dropout_spec* drop,
                      const void* residual, int64_t ldr, void* dx, int64_t lddx, void* workspace, size_t workspace_bytes,
                      fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_linear_dgrad");
    int rc = check_dims(rows, in, out, elem_dtype);
    if (rc) return rc;
    const int es = elem_size(elem_dtype);
    if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU) return FSDP_EINVAL;
    if (rows > 0 && ((rc = check_matrix(dz, out, lddz, es)) || (rc = check_matrix(dx, in, lddx, es)))) return rc;
    if ((rc = check_matrix(w, in, ldw, es))) return rc;
    if (rows > 0 && act != FSDP_ACT_NONE && (rc = check_matrix(preact, in, ldz, es))) return rc;
    if (residual && (rc = check_matrix(residual, in, ldr, es))) return rc;
    if (workspace && !aligned16(workspace)) return FSDP_EALIGN;
    LinProblem p = {};
    if ((rc = make_drop(drop, rows, &p.epi.drop))) return rc;
    if (rows == 0) return FSDP_OK;
    p.mode = kDgrad;
    p.K = out;
    p.planes = elem_dtype == FSDP_F32 ? 3 : 1;
    p.out_bf16 = elem_dtype == FSDP_BF16;
    LinEpi& ep = p.epi;
    ep.out = dx;
    ep.ldo = lddx;
    ep.residual = residual;
    ep.ldr = ldr;
    ep.preact = act != FSDP_ACT_NONE ? const_cast<void*>(preact) : nullptr;
    ep.ldz = ldz;
    ep.rows = rows;
    ep.cols = in;
    ep.act = act;
    ep.vec = std::min({row_class(dx, lddx, es), row_class(residual, ldr, es), row_class(ep.preact, ldz, es)});
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Packer pk{static_cast<unsigned char*>(workspace), workspace_bytes, {}};
    const bool skinny = use_skinny(kDgrad, elem_dtype == FSDP_BF16, rows, in, out);
    if (!skinny && (rc = pk.operand(w, out, in, ldw, elem_dtype, &p.cols_op))) return rc;
    if ((rc = pk.operand(dz, rows, out, lddz, elem_dtype, &p.rows_op))) return rc;
    if (skinny) return run_skinny(kDgrad, elem_dtype, dz, lddz, w, ldw, out, ep, st);
    if (elem_dtype == FSDP_F32 && use_small(kDgrad, rows, in, out))
        return run_small(kDgrad, dz, lddz, w, ldw, out, false, nullptr, ep, st);
    return run_product(p, pk, elem_dtype, st);
}

int fsdp_linear_wgrad(int64_t rows, int64_t in, int64_t out, int32_t elem_dtype, const void* dz, int64_t lddz, const void* x,
                      int64_t ldx, void* dw, int64_t lddw, void* db, int32_t grad_dtype, int32_t accumulate, void* workspace,
                      size_t workspace_bytes, fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_linear_wgrad");
    int rc = check_dims(rows, in, out, elem_dtype);
    if (rc) return rc;
    if (!known(grad_dtype)) return FSDP_EDTYPE;
    const int es = elem_size(elem_dtype), gs = elem_size(grad_dtype);
    if (rows > 0 && ((rc = check_matrix(dz, out, lddz, es)) || (rc = check_matrix(x, in, ldx, es)))) return rc;
    if ((rc = check_matrix(dw, in, lddw, gs)) || (rc = check_vector(db, gs))) return rc;
    if (workspace && !aligned16(workspace)) return FSDP_EALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (accumulate) return FSDP_OK;
        cudaError_t e = cudaMemset2DAsync(dw, size_t(lddw) * gs, 0, size_t(in) * gs, size_t(out), st);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, size_t(out) * gs, st);
        return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "cudaMemset(dw)");
    }
    LinProblem p = {};
    Packer pk{static_cast<unsigned char*>(workspace), workspace_bytes, {}};
    if ((rc = pk.operand(dz, rows, out, lddz, elem_dtype, &p.rows_op)) || (rc = pk.operand(x, rows, in, ldx, elem_dtype, &p.cols_op))) return rc;
    p.mode = kWgrad;
    p.K = rows;
    p.planes = elem_dtype == FSDP_F32 ? 3 : 1;
    p.out_bf16 = grad_dtype == FSDP_BF16;
    LinEpi& ep = p.epi;
    ep.out = dw;
    ep.ldo = lddw;
    ep.rows = out;
    ep.cols = in;
    ep.accumulate = accumulate != 0;
    ep.vec = row_class(dw, lddw, gs);
    ep.db = db;
    // partial sums: room for slabs, always where the sizes allow them
    p.slabs = wgrad_slabs(rows, in, out);
    ep.dz = elem_dtype == FSDP_F32 ? dz : p.rows_op.ptr;
    ep.lddz = elem_dtype == FSDP_F32 ? lddz : p.rows_op.ld;
    ep.dz_rows = rows;
    ep.dz_vec = rows16(ep.dz, ep.lddz, es);
    const int64_t floats = partial_floats(rows, in, out, elem_dtype);
    if (floats) {
        if (!pk.ws || pk.left < size_t(floats * 4)) return FSDP_EINVAL;
        p.partial = reinterpret_cast<float*>(pk.ws);
    }
    if (elem_dtype == FSDP_F32 && use_small(kWgrad, rows, in, out))
        return run_small(kWgrad, dz, lddz, x, ldx, rows, p.out_bf16, p.partial, ep, st);
    return run_product(p, pk, elem_dtype, st);
}

int fsdp_dropout(int64_t rows, int64_t cols, int32_t elem_dtype, const void* x, int64_t ldx, const fsdp_dropout_spec* drop,
                 const void* residual, int64_t ldr, void* y, int64_t ldy, fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_dropout");
    if (!known(elem_dtype)) return FSDP_EDTYPE;
    if (rows < 0 || cols < 0) return FSDP_ESHAPE;
    if (rows > kMaxDim || cols > kMaxDim || rows * cols > kMaxElems) return FSDP_EOVERFLOW;
    Drop d;
    int rc = make_drop(drop, rows, &d);
    if (rc) return rc;
    if (rows == 0 || cols == 0) return FSDP_OK;
    const int es = elem_size(elem_dtype);
    if ((rc = check_matrix(x, cols, ldx, es)) || (rc = check_matrix(y, cols, ldy, es))) return rc;
    if (residual && (rc = check_matrix(residual, cols, ldr, es))) return rc;
    const cudaError_t e = launch_dropout(x, ldx, residual, ldr, y, ldy, elem_dtype == FSDP_BF16, rows, cols, d,
                                         reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FSDP_OK : cuda_fail(e, "k_dropout launch");
}

}  // extern "C"
