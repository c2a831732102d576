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

// A thread: 8 destination columns of one row (a whole 16-byte group; past the last column 0).
template <bool F32>
__global__ void __launch_bounds__(kPackThreads) k_pack(const PackJobs jobs) {
    const int which = blockIdx.x >= jobs.first[1];
    const PackJob& j = jobs.j[which];
    pdl_wait();
    const int64_t groups = j.dld / 8;
    const int64_t i = (int64_t(blockIdx.x) - jobs.first[which]) * kPackThreads + threadIdx.x;
    const int64_t r = i / groups, c = (i - r * groups) * 8;
    if (r >= j.rows) return;
    const int n = j.cols - c >= 8 ? 8 : int(j.cols - c);
    uint16_t* const dst = static_cast<uint16_t*>(j.dst) + r * j.dld + c;
    if constexpr (F32) {
        const float* const p = static_cast<const float*>(j.src) + r * j.ld + c;
        float x[8];
        if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            const float4 a = ld4(p), b = ld4(p + 4);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k] : 0.f;
        }
        uint32_t w[3][4] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t t[3];
            split3(x[k], t);
#pragma unroll
            for (int s = 0; s < 3; ++s) w[s][k / 2] |= t[s] << (16 * (k & 1));
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) stu4(dst + s * j.plane, make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]));
    } else {
        const uint16_t* const p = static_cast<const uint16_t*>(j.src) + r * j.ld + c;
        uint32_t w[4] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k / 2] |= (k < n ? uint32_t(p[k]) : 0u) << (16 * (k & 1));
        stu4(dst, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

}  // namespace

cudaError_t launch_pack(const PackJob* jobs, int n, bool f32, cudaStream_t st) {
    PackJobs pj = {};
    int64_t total = 0;
    for (int k = 0; k < 2; ++k) {
        if (k < n) pj.j[k] = jobs[k];
        pj.first[k] = total;
        if (k < n) total += (jobs[k].rows * (jobs[k].dld / 8) + kPackThreads - 1) / kPackThreads;
    }
    pj.first[2] = total;
    if (n < 2) pj.first[1] = total;
    if (total == 0) return cudaSuccess;
    if (total > INT32_MAX) return cudaErrorInvalidValue;
    return f32 ? launch(k_pack<true>, dim3(unsigned(total)), dim3(kPackThreads), 0, st, pj)
               : launch(k_pack<false>, dim3(unsigned(total)), dim3(kPackThreads), 0, st, pj);
}

}  // namespace fsdp
