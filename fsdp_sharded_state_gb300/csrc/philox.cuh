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

// A dropout as the kernels take it: thr = floor(p * 2^32), scale = fp32(1 / (1 - p)), and
// the ten rounds' keys, which the kernels read as operands from constant memory.
struct Drop {
    uint32_t on, thr;
    float scale;
    uint32_t layer;
    int64_t row0;              // added to the row index of every element
    uint32_t key[10][2];
};

#ifdef __CUDACC__
__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                               const uint32_t (&key)[10][2]) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ key[i][0];
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ key[i][1];
        c3 = uint32_t(a);
    }
    return make_uint4(c0, c1, c2, c3);
}

// The block of columns [4q, 4q + 4) of a row.
__device__ __forceinline__ uint4 drop_words(const Drop& d, int64_t row, int64_t q) {
    const uint64_t r = uint64_t(row + d.row0);
    return philox4x32_10(uint32_t(q), uint32_t(r), uint32_t(r >> 32), d.layer, d.key);
}

// The same blocks over a grid of rows and columns.  While the high word of the row (and so
// the first round's second product) is the same for all of them, the counter enters the
// first three rounds one word at a time: five of their six products depend on the column
// alone or on the row alone, and are shared along the other.  A block then costs 15 products,
// the column's two and the row's one spread over the grid, instead of 20.
struct alignas(16) DropCol {
    uint32_t c3, x0, x2, y3;   // after round 1: word 3; of round 3: what words 0, 2 and 3 take from the column
};
struct DropRow {
    uint32_t h, l;             // round 2's first product: high word with the round's key, low word
};
__device__ __forceinline__ DropCol drop_col(const Drop& d, uint32_t q, uint32_t row_hi) {
    const uint32_t u = 0xCD9E8D57u * row_hi;                     // word 1 after round 1
    const uint64_t a1 = uint64_t(0xD2511F53u) * q;
    const uint64_t b2 = uint64_t(0xCD9E8D57u) * (uint32_t(a1 >> 32) ^ d.layer ^ d.key[0][1]);
    const uint64_t a3 = uint64_t(0xD2511F53u) * (uint32_t(b2 >> 32) ^ u ^ d.key[1][0]);
    return {uint32_t(a1), uint32_t(b2) ^ d.key[2][0], uint32_t(a3 >> 32) ^ d.key[2][1], uint32_t(a3)};
}
// row: its low word; u: the high word of the round constant times the row's high word.
__device__ __forceinline__ DropRow drop_row(const Drop& d, uint32_t row, uint32_t u) {
    const uint64_t a2 = uint64_t(0xD2511F53u) * (u ^ row ^ d.key[0][0]);
    return {uint32_t(a2 >> 32) ^ d.key[1][1], uint32_t(a2)};
}
__device__ __forceinline__ uint4 drop_words(const Drop& d, const DropRow& r, const DropCol& c) {
    const uint64_t b3 = uint64_t(0xCD9E8D57u) * (r.h ^ c.c3);
    uint32_t c0 = uint32_t(b3 >> 32) ^ c.x0, c1 = uint32_t(b3), c2 = c.x2 ^ r.l, c3 = c.y3;
#pragma unroll
    for (int i = 3; i < 10; ++i) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ d.key[i][0];
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ d.key[i][1];
        c3 = uint32_t(a);
    }
    return make_uint4(c0, c1, c2, c3);
}
// A select, not a product with 0: a dropped infinity or NaN becomes 0.
__device__ __forceinline__ float drop1(const Drop& d, uint32_t word, float x) { return word >= d.thr ? x * d.scale : 0.f; }
#endif

}  // namespace fsdp
