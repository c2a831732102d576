// linear_pack.cu -- operands brought into the form that the tensor maps take.
//
// bf16: rows of any alignment and stride copied to rows of whole 16 bytes.
// fp32: x = hi + mid + lo, three bf16 terms of 8 significant bits each (every difference is
// exact in fp32, so the sum is x itself unless x is below 2^-110 or so); a product of two
// such operands keeps the six term products down to 2^-16 of the largest and drops those
// below 2^-24.  An infinity or NaN goes whole into hi, with mid = lo = 0.
#include "common.cuh"
#include "linear.hpp"

namespace fsdp {
namespace {

constexpr int kPackThreads = 256;

struct PackJobs {
    PackJob j[2];
    int64_t first[3];          // first block of each job, and their total
};

// bf16 of x, nearest even, but never an infinity from a finite x.
__device__ __forceinline__ uint32_t term(float x) {
    uint32_t h = to_bf16(x);
    if ((h & 0x7f80u) == 0x7f80u && (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u) h = __float_as_uint(x) >> 16;
    return h;
}

__device__ __forceinline__ void split3(float x, uint32_t (&t)[3]) {
    t[0] = term(x);
    if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) {
        t[1] = t[2] = 0;
        return;
    }
    const float r = x - bf16f(uint16_t(t[0]));
    t[1] = term(r);
    t[2] = term(r - bf16f(uint16_t(t[1])));
}

// The terms of two neighbours, packed.  Values whose high term would round to an infinity, and
// infinities and NaNs themselves, go through split3.
__device__ __forceinline__ void split3_pair(float a, float b, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
    const uint32_t big = 0x7f7f8000u;
    if ((__float_as_uint(a) & 0x7fffffffu) >= big || (__float_as_uint(b) & 0x7fffffffu) >= big) {
        uint32_t x[3], y[3];
        split3(a, x);
        split3(b, y);
        t0 = x[0] | y[0] << 16;
        t1 = x[1] | y[1] << 16;
        t2 = x[2] | y[2] << 16;
        return;
    }
    t0 = pack_bf16x2(a, b);
    a -= bf16lo(t0);
    b -= bf16hi(t0);
    t1 = pack_bf16x2(a, b);
    t2 = pack_bf16x2(a - bf16lo(t1), b - bf16hi(t1));
}

// A thread: 8 destination columns (a whole 16-byte group; past the last column 0) of kPackRows
// rows, their loads first.
constexpr int kPackRows = 4;

template <bool F32>
__global__ void __launch_bounds__(kPackThreads) k_pack(const __grid_constant__ PackJobs jobs) {
    const int which = blockIdx.x >= jobs.first[1];
    const PackJob& j = jobs.j[which];
    pdl_wait();
    const uint32_t groups = uint32_t((j.cols + 7) / 8);
    const int64_t i = (int64_t(blockIdx.x) - jobs.first[which]) * kPackThreads + threadIdx.x;
    const int64_t quad = i / groups, r0 = quad * kPackRows, c = (i - quad * groups) * 8;
    if (r0 >= j.rows) return;
    const int n = j.cols - c >= 8 ? 8 : int(j.cols - c), rows = j.rows - r0 < kPackRows ? int(j.rows - r0) : kPackRows;
    uint16_t* const dst = static_cast<uint16_t*>(j.dst) + r0 * j.dld + c;
    if constexpr (F32) {
        const float* const p = static_cast<const float*>(j.src) + r0 * j.ld + c;
        float x[kPackRows][8];
        const bool vec = n == 8 && ((reinterpret_cast<uintptr_t>(p) | uintptr_t(j.ld * 4)) & 15) == 0;
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) {
            if (r >= rows) break;
            if (vec) {
                const float4 a = ld4(p + r * j.ld), b = ld4(p + r * j.ld + 4);
                x[r][0] = a.x; x[r][1] = a.y; x[r][2] = a.z; x[r][3] = a.w;
                x[r][4] = b.x; x[r][5] = b.y; x[r][6] = b.z; x[r][7] = b.w;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[r][k] = k < n ? p[r * j.ld + k] : 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) {
            if (r >= rows) break;
            uint32_t w[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) split3_pair(x[r][2 * k], x[r][2 * k + 1], w[0][k], w[1][k], w[2][k]);
#pragma unroll
            for (int s = 0; s < 3; ++s) stu4(dst + s * j.plane + r * j.dld, make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]));
        }
    } else {
        const uint16_t* const p = static_cast<const uint16_t*>(j.src) + r0 * j.ld + c;
        uint32_t x[kPackRows][8];
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) {
            if (r >= rows) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[r][k] = k < n ? uint32_t(p[r * j.ld + k]) : 0u;
        }
#pragma unroll
        for (int r = 0; r < kPackRows; ++r) {
            if (r >= rows) break;
            stu4(dst + r * j.dld, make_uint4(x[r][0] | x[r][1] << 16, x[r][2] | x[r][3] << 16, x[r][4] | x[r][5] << 16,
                                             x[r][6] | x[r][7] << 16));
        }
    }
}

}  // namespace

cudaError_t launch_pack(const PackJob* jobs, int n, bool f32, cudaStream_t st) {
    PackJobs pj = {};
    int64_t total = 0;
    for (int k = 0; k < 2; ++k) {
        if (k < n) pj.j[k] = jobs[k];
        pj.first[k] = total;
        if (k < n) total += ((jobs[k].rows + kPackRows - 1) / kPackRows * ((jobs[k].cols + 7) / 8) + kPackThreads - 1) / kPackThreads;
    }
    pj.first[2] = total;
    if (n < 2) pj.first[1] = total;
    if (total == 0) return cudaSuccess;
    if (total > INT32_MAX) return cudaErrorInvalidValue;
    return f32 ? launch(k_pack<true>, dim3(unsigned(total)), dim3(kPackThreads), 0, st, pj)
               : launch(k_pack<false>, dim3(unsigned(total)), dim3(kPackThreads), 0, st, pj);
}

}  // namespace fsdp
