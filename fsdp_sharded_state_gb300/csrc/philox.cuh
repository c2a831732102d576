// philox.cuh -- the counter-based generator of the dropout masks.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products, XORs with a key
// that steps by fixed increments, four 32-bit words out of a 128-bit counter.  A mask
// is never stored: the element at (row, col) of a dropped matrix is kept when word
// col mod 4 of the block with counter (col / 4, row low, row high, layer) and key
// (seed low, seed high) is >= p * 2^32, so forward, recomputation and backward, and
// any split of the rows over calls, meet the same mask.
#pragma once

#include <cstdint>

namespace fsdp {

// A dropout as the kernels take it: thr = floor(p * 2^32), scale = fp32(1 / (1 - p)).
struct Drop {
    uint32_t on, thr;
    float scale;
    uint32_t k0, k1, layer;
    int64_t row0;              // added to the row index of every element
};

#ifdef __CUDACC__
__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                               uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ k0;
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ k1;
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// The block of columns [4q, 4q + 4) of a row.
__device__ __forceinline__ uint4 drop_words(const Drop& d, int64_t row, int64_t q) {
    const uint64_t r = uint64_t(row + d.row0);
    return philox4x32_10(uint32_t(q), uint32_t(r), uint32_t(r >> 32), d.layer, d.k0, d.k1);
}
// A select, not a product with 0: a dropped infinity or NaN becomes 0.
__device__ __forceinline__ float drop1(const Drop& d, uint32_t word, float x) { return word >= d.thr ? x * d.scale : 0.f; }
#endif

}  // namespace fsdp
