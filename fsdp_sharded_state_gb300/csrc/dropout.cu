// dropout.cu -- y = residual + drop(x) over a row-major matrix, the mask drawn where it is
// used (philox.cuh) and never stored; backward is the same call on the gradient.
//
// Bound by HBM bytes (2 or 3 accesses per element) once the generator's integer work, one
// block of about 80 instructions per 4 elements, runs beside the loads.
#include "common.cuh"
#include "linear.hpp"

namespace fsdp {
namespace {

constexpr int kDropThreads = 256;

__device__ __forceinline__ float get(const uint16_t* p) { return bf16f(*p); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// 8 elements, held as they lie in memory.
template <typename T>
struct Pack8 {
    uint4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Pack8<T> read8(const T* p) {
    Pack8<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) r.q[i] = ldu4(reinterpret_cast<const char*>(p) + 16 * i);
    return r;
}
__device__ __forceinline__ float elem(const Pack8<uint16_t>& r, int i) {
    const uint32_t w = i / 2 == 0 ? r.q[0].x : i / 2 == 1 ? r.q[0].y : i / 2 == 2 ? r.q[0].z : r.q[0].w;
    return i & 1 ? bf16hi(w) : bf16lo(w);
}
__device__ __forceinline__ float elem(const Pack8<float>& r, int i) {
    const uint4 q = r.q[i / 4];
    return __uint_as_float((i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w);
}
__device__ __forceinline__ void write8(uint16_t* p, const float (&v)[8]) {
    stu4(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}
__device__ __forceinline__ void write8(float* p, const float (&v)[8]) {
    st4(p, make_float4(v[0], v[1], v[2], v[3]));
    st4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}

// Rows of whole, aligned groups of 8 elements: a thread takes one group of kDropRows
// consecutive rows, all loads first, and the generator's column products once.  `rows` all
// share the high word of row0 + row.
constexpr int kDropRows = 4;

template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads)
k_dropout8(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy, int64_t rows, uint32_t groups,
           const __grid_constant__ Drop d) {
    pdl_wait();
    const int64_t i = int64_t(blockIdx.x) * kDropThreads + threadIdx.x;
    const int64_t quad = i / groups, row0 = quad * kDropRows;
    const uint32_t g = uint32_t(i - quad * groups);
    if (row0 >= rows) return;
    const int n = rows - row0 < kDropRows ? int(rows - row0) : kDropRows;
    const T* px = x + row0 * ldx + int64_t(g) * 8;
    const T* pr = RES ? res + row0 * ldr + int64_t(g) * 8 : nullptr;
    T* py = y + row0 * ldy + int64_t(g) * 8;
    Pack8<T> a[kDropRows], b[kDropRows];
#pragma unroll
    for (int k = 0; k < kDropRows; ++k) {
        if (k < n) {
            a[k] = read8(px + k * ldx);
            if constexpr (RES) b[k] = read8(pr + k * ldr);
        }
    }
    const uint64_t r = uint64_t(row0 + d.row0);
    const uint32_t u = __umulhi(0xCD9E8D57u, uint32_t(r >> 32));
    const DropCol c0 = drop_col(d, 2 * g, uint32_t(r >> 32)), c1 = drop_col(d, 2 * g + 1, uint32_t(r >> 32));
#pragma unroll
    for (int k = 0; k < kDropRows; ++k) {
        if (k >= n) break;
        uint4 w[2] = {};
        if (d.on) {
            const DropRow dr = drop_row(d, uint32_t(r) + k, u);
            w[0] = drop_words(d, dr, c0);
            w[1] = drop_words(d, dr, c1);
        }
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[4 * h] = drop1(d, w[h].x, elem(a[k], 4 * h));
            v[4 * h + 1] = drop1(d, w[h].y, elem(a[k], 4 * h + 1));
            v[4 * h + 2] = drop1(d, w[h].z, elem(a[k], 4 * h + 2));
            v[4 * h + 3] = drop1(d, w[h].w, elem(a[k], 4 * h + 3));
        }
        if constexpr (RES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += elem(b[k], e);
        }
        write8(py + k * ldy, v);
    }
}

__device__ __forceinline__ uint32_t keep8(const Drop& d, int64_t row, int64_t chunk) {
    const uint4 a = drop_words(d, row, 2 * chunk), b = drop_words(d, row, 2 * chunk + 1);
    return uint32_t(a.x >= d.thr) | uint32_t(a.y >= d.thr) << 1 | uint32_t(a.z >= d.thr) << 2 | uint32_t(a.w >= d.thr) << 3 |
           uint32_t(b.x >= d.thr) << 4 | uint32_t(b.y >= d.thr) << 5 | uint32_t(b.z >= d.thr) << 6 | uint32_t(b.w >= d.thr) << 7;
}

// Rows that start at any element, in step: x, residual and y of a row have the same address
// modulo 16 bytes (contiguous matrices of one odd width).  With m elements before a row's
// first 16-byte boundary rounded down, lane G holds columns [8G - m, 8G - m + 8): an aligned
// group whose keep bits are the upper m of chunk G - 1 (columns 8G - 8 on) and the lower 8 - m
// of chunk G, so a lane draws one chunk and takes the other from its neighbour; the first
// lane only draws.
constexpr int kStepGroups = 31;

template <typename T>
__global__ void __launch_bounds__(kDropThreads)
k_dropout_step(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy, int64_t rows, int64_t cols, int64_t strips,
               const __grid_constant__ Drop d) {
    constexpr int E = 16 / sizeof(T);
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t i = int64_t(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5);
    const int64_t r = i / strips, s = i - r * strips;
    if (r >= rows) return;
    T* const py = y + r * ldy;
    const int m = int(reinterpret_cast<uintptr_t>(py) / sizeof(T)) & (E - 1);
    const int64_t G = s * kStepGroups + lane - 1, c = 8 * G - m;          // this lane's chunk; its group's first column
    const int64_t lo = c < 0 ? 0 : c, hi = c + 8 < cols ? c + 8 : cols;
    const bool mine = lane > 0 && lo < hi, whole = mine && hi - lo == 8;
    const T* const px = x + r * ldx;
    const T* const pr = res ? res + r * ldr : nullptr;
    Pack8<T> a = {}, b = {};
    if (whole) {
        a = read8(px + c);
        if (pr) b = read8(pr + c);
    }
    const uint32_t chunk = d.on && G >= 0 && 8 * G < cols ? keep8(d, r, G) : 0xffu;
    const uint32_t before = __shfl_up_sync(0xffffffffu, chunk, 1);
    const uint32_t keep = (chunk << 8 | before) >> (8 - m);                // bit e: column c + e
    if (whole) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = keep >> e & 1 ? elem(a, e) * d.scale : 0.f;
        if (pr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += elem(b, e);
        }
        write8(py + c, v);
    } else if (mine) {
        for (int64_t k = lo; k < hi; ++k) {
            float v = keep >> int(k - c) & 1 ? get(px + k) * d.scale : 0.f;
            if (pr) v += get(pr + k);
            put(py + k, v);
        }
    }
}

// Any alignment: a warp covers 256 columns of a row; a lane draws the generator's blocks of
// 8 columns, reads and writes columns 32 apart, and fetches its words from the lanes that
// drew them as keep bits.
constexpr int kDropCols = 256;

template <typename T>
__global__ void __launch_bounds__(kDropThreads)
k_dropout1(const T* x, int64_t ldx, const T* res, int64_t ldr, T* y, int64_t ldy, int64_t rows, int64_t cols, int64_t strips,
           const __grid_constant__ Drop d) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t i = int64_t(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5);
    const int64_t r = i / strips, s = i - r * strips;
    if (r >= rows) return;
    const int64_t c0 = s * kDropCols + lane;
    const T* px = x + r * ldx + c0;
    const T* pr = res ? res + r * ldr + c0 : nullptr;
    T* py = y + r * ldy + c0;
    const int n = cols - c0 > 224 ? 8 : cols > c0 ? int((cols - c0 + 31) >> 5) : 0;   // of this lane's columns
    float v[8], t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        v[k] = k < n ? get(px + 32 * k) : 0.f;
        t[k] = pr && k < n ? get(pr + 32 * k) : 0.f;
    }
    uint32_t keep = 0xff;                          // of columns 8 lane .. 8 lane + 7 of the strip
    if (d.on) {
        keep = keep8(d, r, s * (kDropCols / 8) + lane);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // column 32 k + lane of the strip: bit lane mod 8 of lane 4 k + lane / 8
        const uint32_t bits = __shfl_sync(0xffffffffu, keep, 4 * k + (lane >> 3));
        if (k < n) {
            float o = bits >> (lane & 7) & 1 ? v[k] * d.scale : 0.f;
            if (pr) o += t[k];
            put(py + 32 * k, o);
        }
    }
}

template <typename T>
cudaError_t run(const void* x, int64_t ldx, const void* res, int64_t ldr, void* y, int64_t ldy, int64_t rows, int64_t cols,
                const Drop& d0, cudaStream_t st) {
    Drop d = d0;
    if (!d.on) {                                   // a mask that keeps all: thr = 0 <= every word
        d.thr = 0;
        d.scale = 1.f;
    }
    const T *px = static_cast<const T*>(x), *pr = static_cast<const T*>(res);
    T* py = static_cast<T*>(y);
    constexpr int64_t E = 16 / sizeof(T);
    auto phase = [](const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; };
    auto same = [&](const void* p, int64_t ld) { return !p || (phase(p) == phase(y) && (rows == 1 || (ld - ldy) % E == 0)); };
    const bool step = same(x, ldx) && same(res, ldr);
    if (step && phase(y) == 0 && (rows == 1 || ldy % E == 0) && cols % 8 == 0) {
        // rows up to the next change of the row's high word at a time (all of them, in practice)
        for (int64_t r = 0; r < rows;) {
            const int64_t to_edge = (int64_t(1) << 32) - ((d.row0 + r) & 0xffffffffLL);
            const int64_t n = rows - r < to_edge ? rows - r : to_edge;
            const int64_t blocks = ((n + kDropRows - 1) / kDropRows * (cols / 8) + kDropThreads - 1) / kDropThreads;
            if (blocks > INT32_MAX) return cudaErrorInvalidValue;
            Drop dr = d;
            dr.row0 += r;
            const T* const rr = pr ? pr + r * ldr : nullptr;
            const cudaError_t e =
                pr ? launch(k_dropout8<T, true>, dim3(unsigned(blocks)), dim3(kDropThreads), 0, st, px + r * ldx, ldx, rr, ldr,
                            py + r * ldy, ldy, n, uint32_t(cols / 8), dr)
                   : launch(k_dropout8<T, false>, dim3(unsigned(blocks)), dim3(kDropThreads), 0, st, px + r * ldx, ldx, rr, ldr,
                            py + r * ldy, ldy, n, uint32_t(cols / 8), dr);
            if (e != cudaSuccess) return e;
            r += n;
        }
        return cudaSuccess;
    }
    // a strip per warp: of 31 groups of 8 columns shifted by up to E - 1, or of 256 columns
    const int64_t strips = step ? ((cols + E - 1 + 7) / 8 + kStepGroups - 1) / kStepGroups : (cols + kDropCols - 1) / kDropCols;
    const int64_t per = kDropThreads / 32, blocks = (rows * strips + per - 1) / per;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return step ? launch(k_dropout_step<T>, dim3(unsigned(blocks)), dim3(kDropThreads), 0, st, px, ldx, pr, ldr, py, ldy, rows,
                         cols, strips, d)
                : launch(k_dropout1<T>, dim3(unsigned(blocks)), dim3(kDropThreads), 0, st, px, ldx, pr, ldr, py, ldy, rows, cols,
                         strips, d);
}

}  // namespace

cudaError_t launch_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy, bool bf16,
                           int64_t rows, int64_t cols, const Drop& d, cudaStream_t st) {
    return bf16 ? run<uint16_t>(x, ldx, residual, ldr, y, ldy, rows, cols, d, st)
                : run<float>(x, ldx, residual, ldr, y, ldy, rows, cols, d, st);
}

}  // namespace fsdp
