// ns_api.cu -- Newton-Schulz steps: their scales, their workspace, their launches and the extern
// "C" entry points.  Every check runs before the first launch.
#include <algorithm>
#include <cmath>

#include "internal.hpp"
#include "ns.hpp"

namespace fsdp {
namespace {

// a, b, c of the quintic that takes singular values from [0.01, 1] to about 0.7 ... 1.2 in five
// steps (Jordan et al., "Muon: an optimizer for hidden layers in neural networks", 2024).
constexpr float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Largest |p(s)|, p(s) = a s + b s^3 + c s^5, and |q(t)|, q(t) = a + b t + c t^2, for s in [0, u], t = s^2.
void step_bounds(double a, double b, double c, double u, double* p, double* q) {
    auto gain = [&](double t) { return a + t * (b + t * c); };
    auto val = [&](double t) { return std::sqrt(t) * gain(t); };
    const double top = u * u;
    *p = std::fabs(val(top));
    *q = std::max(std::fabs(gain(0)), std::fabs(gain(top)));
    auto at = [&](double t) {
        if (t > 0 && t < top) {
            *p = std::max(*p, std::fabs(val(t)));
            *q = std::max(*q, std::fabs(gain(t)));
        }
    };
    if (c != 0) {
        const double d = 9 * b * b - 20 * a * c;       // p' = a + 3 b t + 5 c t^2
        if (d >= 0) {
            at((-3 * b + std::sqrt(d)) / (10 * c));
            at((-3 * b - std::sqrt(d)) / (10 * c));
        }
        at(-b / (2 * c));
    } else if (b != 0) {
        at(-a / (3 * b));
    }
}

// The power of two that brings values of up to `bound` to at most 2^15, half of fp16's range, but
// values of up to 1 no further than 2^15.
float scale_of(double bound) { return float(std::ldexp(1.0, 15 - std::max(0, int(std::ceil(std::log2(std::max(bound, 1.0))))))); }

}  // namespace

bool ns_scales(const float* coeffs, int steps, NsScales* s) {
    double u = 1.0;
    s->x[0] = scale_of(u);
    for (int k = 0; k < steps; ++k) {
        const float* const f = coeffs ? coeffs + 3 * k : kDefault;
        if (!std::isfinite(f[0]) || !std::isfinite(f[1]) || !std::isfinite(f[2])) return false;
        double p, q;
        step_bounds(f[0], f[1], f[2], u, &p, &q);
        if (!(p <= 4.0) || !(q <= 1024.0)) return false;
        s->a[k] = scale_of(u * u);
        s->b[k] = scale_of(q);
        u = p;
        s->x[k + 1] = scale_of(u);
    }
    return true;
}

NsWork ns_work(int64_t rows, int64_t cols, int64_t count) {
    NsWork w;
    w.m = std::min(rows, cols);
    w.n = std::max(rows, cols);
    const int64_t mp = round_up(w.m, 256), np = round_up(w.n, 256);
    // enough matrices at once to fill the device several times over, in 256 MB of planes or one matrix
    w.chunk = int(std::max<int64_t>(1, std::min<int64_t>({count, kNsMaxBatch, (int64_t(1) << 26) / (mp * np)})));
    w.x0 = 0;
    w.x1 = w.x0 + w.chunk * mp * np * 4;
    w.a = w.x1 + w.chunk * mp * np * 4;
    w.b = w.a + w.chunk * mp * mp * 4;
    w.partial = w.b + w.chunk * mp * mp * 4;
    w.end = w.partial + int64_t(w.chunk) * kNsMaxParts * 8;
    return w;
}

cudaError_t ns_run(const NsWork& w, unsigned char* ws, int batch, const NsMatrices& src, const NsMatrices& dst, int parts, float eps,
                   const float* coeffs, int steps, const NsScales& sc, cudaStream_t st) {
    const int64_t mp = round_up(w.m, 256), np = round_up(w.n, 256);
    auto planes = [&](int64_t at, int64_t cols, int64_t ld) {
        return NsPlanes{reinterpret_cast<uint16_t*>(ws + at), w.m, cols, ld, mp * ld};
    };
    NsPlanes x = planes(w.x0, w.n, np), next = planes(w.x1, w.n, np);
    const NsPlanes a = planes(w.a, w.m, mp), b = planes(w.b, w.m, mp);
    cudaError_t e = launch_ns_pack(src, batch, x, reinterpret_cast<const double*>(ws + w.partial), parts, sc.x[0], eps, st);
    for (int k = 0; k < steps && e == cudaSuccess; ++k) {
        const float* const f = coeffs ? coeffs + 3 * k : kDefault;
        const float sx = sc.x[k], sa = sc.a[k], sb = sc.b[k];      // powers of two
        NsProduct p = {};
        p.batch = batch;
        p.kind = kNsGram;
        p.x = x;
        p.out = a;
        p.alpha = sa / (sx * sx);
        if ((e = launch_ns_gram(p, st)) != cudaSuccess) break;
        p.kind = kNsPoly;
        p.x = a;
        p.out = b;
        p.alpha = f[2] * (sb / (sa * sa));
        p.beta = f[1] * (sb / sa);
        p.diag = f[0] * sb;
        if ((e = launch_ns_poly(p, st)) != cudaSuccess) break;
        p.x = b;
        p.y = x;
        if (k + 1 < steps) {
            p.kind = kNsStep;
            p.out = next;
            p.alpha = sc.x[k + 1] / (sb * sx);
            e = launch_ns_step(p, st);
            std::swap(x, next);
        } else {
            p.kind = kNsLast;
            p.last = &dst;
            p.alpha = 1.f / (sb * sx);
            e = launch_ns_last(p, st);
        }
    }
    return e;
}

}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::detail;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxElems = int64_t(1) << 34;              // of a matrix, padded

bool known(int32_t dtype) { return dtype == FSDP_F32 || dtype == FSDP_BF16; }

int check_dims(int64_t count, int64_t rows, int64_t cols) {
    if (count < 0 || rows < 1 || cols < 1) return FSDP_ESHAPE;
    if (rows > kMaxDim || cols > kMaxDim) return FSDP_EOVERFLOW;
    if (round_up(rows, 256) * round_up(cols, 256) > kMaxElems) return FSDP_EOVERFLOW;
    return FSDP_OK;
}

}  // namespace

extern "C" {

size_t fsdp_newton_schulz_workspace_bytes(int32_t count, int64_t rows, int64_t cols) {
    if (check_dims(count, rows, cols) || count == 0) return 0;
    return size_t(ns_work(rows, cols, count).end);
}

int fsdp_newton_schulz(int32_t count, int64_t rows, int64_t cols, const void* const* src, const int64_t* ld_src, int32_t src_dtype,
                       void* const* dst, const int64_t* ld_dst, int32_t dst_dtype, int32_t steps, const float* coeffs, float eps,
                       void* workspace, size_t workspace_bytes, fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_newton_schulz");
    int rc = check_dims(count, rows, cols);
    if (rc) return rc;
    if (!known(src_dtype) || !known(dst_dtype)) return FSDP_EDTYPE;
    if (steps < 1 || steps > kNsMaxSteps || !(eps > 0.f) || !std::isfinite(eps)) return FSDP_EINVAL;
    NsScales sc;
    if (!ns_scales(coeffs, steps, &sc)) return FSDP_EINVAL;
    if (count == 0) return FSDP_OK;
    if (!src || !dst || !ld_src || !ld_dst) return FSDP_EINVAL;
    const unsigned se = src_dtype == FSDP_F32 ? 4 : 2, de = dst_dtype == FSDP_F32 ? 4 : 2;
    for (int32_t i = 0; i < count; ++i) {
        if (!src[i] || !dst[i]) return FSDP_EINVAL;
        if (reinterpret_cast<uintptr_t>(src[i]) % se || reinterpret_cast<uintptr_t>(dst[i]) % de) return FSDP_EALIGN;
        if (ld_src[i] < cols || ld_dst[i] < cols) return FSDP_ESHAPE;
        if (ld_src[i] > INT32_MAX || ld_dst[i] > INT32_MAX) return FSDP_EOVERFLOW;
    }
    const NsWork w = ns_work(rows, cols, count);
    if (!workspace || workspace_bytes < size_t(w.end)) return FSDP_EINVAL;
    if (!aligned16(workspace)) return FSDP_EALIGN;
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int parts = ns_parts(rows * cols);
    for (int32_t first = 0; first < count; first += w.chunk) {
        const int n = std::min<int>(w.chunk, count - first);
        NsMatrices s = {}, d = {};
        for (int i = 0; i < n; ++i) {
            s.p[i] = const_cast<void*>(src[first + i]);
            s.ld[i] = ld_src[first + i];
            d.p[i] = dst[first + i];
            d.ld[i] = ld_dst[first + i];
        }
        s.tall = d.tall = rows > cols ? ~uint64_t(0) : 0;
        s.bf16 = src_dtype == FSDP_BF16;
        d.bf16 = dst_dtype == FSDP_BF16;
        cudaError_t e = launch_ns_squares(s, n, w.m, w.n, reinterpret_cast<double*>(ws + w.partial), parts, st);
        if (e != cudaSuccess) return cuda_fail(e, "k_ns_squares launch");
        e = ns_run(w, ws, n, s, d, parts, eps, coeffs, steps, sc, st);
        if (e != cudaSuccess) return cuda_fail(e, "k_ns launch");
    }
    return FSDP_OK;
}

}  // extern "C"
