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
    s->top[0] = u;
    for (int k = 0; k < steps; ++k) {
        const float* const f = coeffs ? coeffs + 3 * k : kDefault;
        if (!std::isfinite(f[0]) || !std::isfinite(f[1]) || !std::isfinite(f[2])) return false;
        double p, q;
        step_bounds(f[0], f[1], f[2], u, &p, &q);
        if (!(p <= 4.0) || !(q <= 1024.0)) return false;
        s->a[k] = scale_of(u * u);
        s->b[k] = scale_of(q);
        s->gain[k] = q;
        u = p;
        s->top[k + 1] = u;
        s->x[k + 1] = scale_of(u);
    }
    return true;
}

NsWork ns_work(int64_t rows, int64_t cols, int64_t count) {
    NsWork w;
    w.m = std::min(rows, cols);
    w.n = std::max(rows, cols);
    if (use_ns_tiny(w.m, w.n)) {
        w.chunk = int(std::max<int64_t>(1, std::min<int64_t>(count, kNsMaxBatch)));
        w.x0 = w.x1 = w.square[0] = w.square[1] = w.square[2] = w.square[3] = w.partial = 0;
        w.end = int64_t(w.chunk) * kNsMaxParts * 4;
        return w;
    }
    const int64_t mp = round_up(w.m, 256), np = round_up(w.n, 256);
    // enough matrices at once to fill the device several times over, in 256 MB of planes or one matrix
    w.chunk = int(std::max<int64_t>(1, std::min<int64_t>({count, kNsMaxBatch, (int64_t(1) << 26) / (mp * np)})));
    w.x0 = 0;
    w.x1 = w.x0 + w.chunk * mp * np * 4;
    for (int i = 0; i < 4; ++i) w.square[i] = w.x1 + w.chunk * (mp * np + i * mp * mp) * 4;
    w.partial = w.square[3] + w.chunk * mp * mp * 4;
    w.end = w.partial + int64_t(w.chunk) * kNsMaxParts * 4;
    return w;
}

// Steps one by one cost a pass over X each for A = X X^T and for X' = B X.  A step that follows
// another can do without: with B_0 from A_0 = X X^T, the next A is B_0 A_0 B_0 and the next B_1 a polynomial of
// it, and X takes both as (B_1 B_0) X.  That is three products of m x m in place of m x m x n and
// m x n x m, less work where n > m: 4096 x 11008 takes 30 units of m^3 for five steps in groups
// of 3 and 2 instead of 45, 4.2 instead of 5.9 ms; 2048 x 5504 0.61 instead of 0.84.
//
// What it costs in precision.  An error d of A grows by up to the square of the first coefficient (11.9)
// with each step that A is carried on, and comes into B times the second: 680 d after two steps, 1.6e-4 of
// the norm for d = 2^-22.  Where A is computed anew each time, X keeps the digits of its own columns, large or
// small: measured against 64 bits, in 1e-6 of the result's norm (in brackets fp32 products one step at a time), 1024 x 4096
// noise takes 3.5 in groups of three and 1.2 one by one (3.8), but with all columns except four made 10^-4 of
// these 38 and 3.3 (2.2).  So groups are for results that need fewer digits (`groups`):
//   - bf16 ones, rounded by up to 2^-8 of each element;
//   - the Muon step's, which are added to weights: a matrix that few columns hold has a small result, of
//     which 38 are 8.3e-5 in absolute terms, below what fp32 products leave of the noise (1.2e-4).
// fp32 results of fsdp_newton_schulz go one by one.
//
// Small and long matrices have more of their directions where groups lose: measured on noise with four strong directions
// (fp32 products 1.3 at m = 128 to 3.6 at 1024), groups of three 4.9 to 15 at m = 128 to 256, 3.7 to 6 at
// 384 and 448, 2.1 to 3.4 at 768, 2.0 to 2.8 from 1024 on; groups of two 1.3 to 3.3 where n >= 3 m, 2.4 to 3.8 below,
// and up to 3.2 at m = 24 and 32; steps one by one 0.7 to 2.9 (1.8 there).  So three steps from 768 on, two from 64
// on where n >= 3 m, and a product of gains that leaves the others' digits (kGroupGain).
int group_steps(int64_t m, int64_t n) { return m >= 768 ? 3 : m >= 64 && n >= 3 * m ? 2 : 1; }
constexpr double kGroupGain = 64.0;

// What the accumulators' rounding towards zero takes on average: measured 2.6e-7 of X X^T, whose
// diagonal adds up 16 equal shares a K step, 1.2e-7 of products of symmetric ones, whose diagonals hold
// most of a sum in one term (and 0.6e-7 of Q X, left as it is).  Given back here, since the
// polynomials' cancelling terms answer it with about ten times as much: eight 256 x 1024 matrices
// 3.1e-6 -> 2.4e-6 off.
//
// The mean is that of sums whose terms are alike.  A matrix whose mass lies in few K steps, or in 16 columns
// of them, loses less; measured over nine kinds of matrices (noise, one spectrum or another, mass in 64 columns, in 16, in
// 16 of every 64, on the diagonal) and nine sizes, results are 0.5 to 1.1 times as far off as without, and up to 1.4
// times where 16 columns hold all (256 x 256 1.0e-6 -> 1.3e-6, 1024 x 1024 1.0e-6 -> 1.4e-6; fp32 products 1.4e-6 and 2.1e-6).
constexpr float kGramBack = 1.f + 0x1p-22f, kSquareBack = 1.f + 0x1p-23f;

cudaError_t ns_run(const NsWork& w, unsigned char* ws, int batch, const NsMatrices& src, const NsMatrices& dst, int parts, float eps,
                   const float* coeffs, int steps, const NsScales& sc, bool groups, cudaStream_t st) {
    if (use_ns_tiny(w.m, w.n)) return launch_ns_tiny(src, dst, batch, w.m, w.n, eps, coeffs, steps, kDefault, st);
    const int64_t mp = round_up(w.m, 256), np = round_up(w.n, 256);
    auto planes = [&](int64_t at, int64_t cols, int64_t ld) {
        return NsPlanes{reinterpret_cast<uint16_t*>(ws + at), w.m, cols, ld, mp * ld};
    };
    NsPlanes x = planes(w.x0, w.n, np), next = planes(w.x1, w.n, np), sq[4];
    for (int i = 0; i < 4; ++i) sq[i] = planes(w.square[i], w.m, mp);
    NsProduct p = {};
    p.batch = batch;
    p.x = p.y = x;
    const float over_x = cost_ns_gram(p);
    p.x = p.y = sq[0];
    const float square = cost_ns_mul(p);
    p.y = x;
    const int most = groups && over_x + cost_ns_step(p) > 3.f * square ? group_steps(w.m, w.n) : 1;
    cudaError_t e = launch_ns_pack(src, batch, x, reinterpret_cast<const float*>(ws + w.partial), parts, sc.x[0], eps, st);
    for (int k = 0; k < steps && e == cudaSuccess;) {
        // this group: steps k .. k + n, as even as they go
        const int left = steps - k, room = (left + most - 1) / most;
        int n = (left + room - 1) / room;
        double gain = 1.0;
        for (int j = 0; j < n; ++j) {
            gain *= sc.gain[k + j];
            if (j > 0 && gain > kGroupGain) n = j;
        }
        // where A, B and Q lie among the four square buffers
        int a = 0, b = 1, q = 1;
        auto other = [](int i, int j, int l) {
            int f = 0;
            while (f == i || f == j || f == l) ++f;
            return f;
        };
        auto product = [&](cudaError_t (*launch)(const NsProduct&, cudaStream_t), int i, int j, int out, float alpha) {
            p.x = sq[i];
            p.y = sq[j];
            p.out = sq[out];
            p.alpha = alpha;
            if (e == cudaSuccess) e = launch(p, st);
        };
        float sq_q = sc.b[k];                    // Q's scale; every scale is a power of two
        gain = 1.0;
        for (int j = 0; j < n; ++j) {
            const float* const f = coeffs ? coeffs + 3 * (k + j) : kDefault;
            const float sa = sc.a[k + j], sb = sc.b[k + j];
            if (j == 0) {
                p.x = x;
                p.out = sq[a];
                p.alpha = kGramBack * (sa / (sc.x[k] * sc.x[k]));
                if (e == cudaSuccess) e = launch_ns_gram(p, st);
            } else {                             // C = B A, A = C B; the old B is not needed any more, unless it is Q
                const float s0 = sc.b[k + j - 1], s1 = sc.a[k + j - 1], s2 = scale_of(sc.top[k + j - 1] * sc.top[k + j]);
                const int c = other(a, b, q);
                product(launch_ns_mul, b, a, c, kSquareBack * (s2 / (s0 * s1)));
                product(launch_ns_mul, c, b, a, kSquareBack * (sa / (s2 * s0)));
                b = other(a, q, q);
            }
            p.beta = f[1] * (sb / sa);
            p.diag = f[0] * sb;
            product(launch_ns_poly, a, a, b, kSquareBack * f[2] * (sb / (sa * sa)));
            gain *= sc.gain[k + j];
            if (j > 0) {                         // Q = B Q
                const float s = scale_of(gain);
                const int to = other(a, b, q);
                product(launch_ns_mul, b, q, to, kSquareBack * (s / (sb * sq_q)));
                q = to;
                sq_q = s;
            }
        }
        if (e != cudaSuccess) break;
        k += n;
        p.x = sq[q];
        p.y = x;
        if (k < steps) {
            p.out = next;
            p.alpha = sc.x[k] / (sq_q * sc.x[k - n]);
            e = launch_ns_step(p, st);
            std::swap(x, next);
        } else {
            p.last = &dst;
            p.alpha = 1.f / (sq_q * sc.x[k - n]);
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
    if (steps < 1 || steps > kNsMaxSteps || !(eps >= kNsLeastEps) || !std::isfinite(eps)) return FSDP_EINVAL;
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
        cudaError_t e = cudaSuccess;
        if (!use_ns_tiny(w.m, w.n)) e = launch_ns_squares(s, n, w.m, w.n, reinterpret_cast<float*>(ws + w.partial), parts, st);
        if (e != cudaSuccess) return cuda_fail(e, "k_ns_squares launch");
        e = ns_run(w, ws, n, s, d, parts, eps, coeffs, steps, sc, dst_dtype == FSDP_BF16, st);
        if (e != cudaSuccess) return cuda_fail(e, "k_ns launch");
    }
    return FSDP_OK;
}

}  // extern "C"
