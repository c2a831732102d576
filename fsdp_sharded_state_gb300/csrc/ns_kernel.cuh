// ns_kernel.cuh -- the matrix products of Newton-Schulz steps (sm_103a).
//
// D[M, N] = sum over k of A[M, k] B[N, k] for a batch of matrices of one shape, on the 5th-generation
// tensor cores, both operands fp32 values held as two fp16 terms.
//
// Precision.  A step multiplies what lies in small singular directions by up to its first
// coefficient, five steps of the usual ones by 485: roundings of the first X come out that much
// larger, so one 16-bit term is not enough for an fp32 result (and costs a bf16 one more than its own
// rounding).  Two fp16 terms hold 22 significant bits (hi rounded to nearest, lo = the rest rounded);
// the operands are scaled by powers of two so that no value of the schedule exceeds 2^15 and lo
// keeps its digits down to 2^-24 of 1.  Three products hi hi + hi lo + lo hi drop 2^-22 of each
// product: what fp32 products round.  The tensor cores round their accumulators towards zero
// at every step, which shrinks all of a product alike, and the steps' polynomials, whose terms
// cancel, answer a common 4e-7 of every product with 4e-6 to 1e-5 of the result (chunks of four
// K steps did).  So the accumulators are emptied into fp32 registers at every K step of 64, small
// products first: four additions round at the full sum's size.
//
// Work.  X X^T and A A are symmetric: only tiles at or below the diagonal are computed, and what
// lies off the diagonal's square is stored twice, as it is and mirrored (a lane holds a row, so the
// mirrored row is 32 consecutive elements of a warp).  B X needs X along its columns, which the
// matrix descriptors take as an MN-major operand: nothing is transposed in memory, and a I is
// in B's diagonal, so that no epilogue but poly's reads anything.  Several steps can share one pass over
// X (ns_run): all in between are products of polynomials of one symmetric matrix, lower tiles too.
//
// Roles of a CTA (12 warps) as in the linear layers' kernel: warp 8 loads the operand tiles with
// tensor-map copies into a ring of stages, warp 9 issues the MMAs, warps 0-7 empty the double-buffered
// accumulators and store.  Pairs of CTAs (cta_group::2) share the B operand of 256 x 256 tiles: 64 KB
// of stage for 1536 clocks of MMA.  Sizes with too few such tiles take 256 x 128, or tiles of one CTA
// of 128 x 64 with K split over a cluster and joined in shared memory in a fixed order.  At 4096 x 11008
// the three kinds of products run at 1.5 (m x m x m), 1.69 (X X^T) and 1.73 PFLOP/s (B X) of fp16
// operations, the last two at the rate that the power limit leaves a library product.
//
// Every wait on an mbarrier is bounded; a role that gives up records it (g_wait_error of this
// translation unit, read by fsdp_check_status), lets copies in flight land and goes to the
// teardown, which every thread of the CTA (and of the cluster) reaches on every path.
#pragma once

#include <cuda_fp16.h>

#include "internal.hpp"
#include "ns.hpp"
#include "tc5.cuh"

namespace fsdp {
namespace {

constexpr int kNsEpiWarps = 8, kNsThreads = 384;
constexpr int kNsMaxStages = 8;
constexpr int kUnitLd = 36;                     // floats of a row of a 32 x 32 unit in shared memory
constexpr int kUnitFloats = 32 * kUnitLd;

// ---- two fp16 terms ----------------------------------------------------------------
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ float2 join2(uint32_t hi, uint32_t lo) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    return make_float2(h.x + l.x, h.y + l.y);
}

template <int EP_, int CG_, int BN_, bool SPLIT_>
struct NsCfg {
    static constexpr int EP = EP_, CG = CG_, BN = BN_;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr bool TRI = EP != kNsStep && EP != kNsLast;  // symmetric: lower tiles only
    static constexpr bool B_MN = !TRI;
    static constexpr int TM = 128 * CG, R = TM / BN;             // R tiles side by side make a square
    static constexpr int BROWS = BN / CG;
    static constexpr bool CUT = CG == 2 && BN == 256;            // tiles of the last wave may be halved
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BROWS * 128;
    static constexpr int STAGE = 2 * (A_BYTES + B_BYTES);
    static constexpr int JOIN = SPLIT ? BN / 8 * kUnitFloats * 4 : 0;
    static constexpr int MORE = 2048;                            // alignment, barriers
    static constexpr int FIT = (227 * 1024 - MORE - JOIN) / STAGE;
    static constexpr int STAGES = FIT < kNsMaxStages ? FIT : kNsMaxStages;
    static constexpr int SMEM = STAGES * STAGE + JOIN + MORE;
    static constexpr int TMEM = 2 * BN;
    static constexpr bool REGS = CG == 2;                        // see setmaxnreg below
    static_assert(R * BN == TM, "a tile's columns divide its rows");
    static_assert(STAGES >= 2 && SMEM > 114 * 1024 && SMEM <= 227 * 1024, "one CTA per SM: its TMEM is never contended");
    static_assert(!SPLIT || CG == 1, "a cluster is a pair or a split");
};

// Tiles of one matrix (`per`), of which a symmetric product has the lower ones only; the first
// `whole` tiles of the batch are worked on as they are, the others in halves of 128 columns.
struct NsShape {
    int32_t m_tiles, n_tiles, n_kb, splits, per, batch, whole;
};

struct NsEpi {
    uint16_t* out;
    int64_t ldo, plane;
    const uint16_t* in;                         // poly: A
    float alpha, beta, diag;
    int32_t rows, cols;                         // last: of the result
};
struct NsNoLast {};

// What becomes of 32 columns from `col` of row `row` of matrix `mat` (a lane's own row).
template <class C, class Last>
__device__ __forceinline__ void ns_emit(const NsEpi& ep, const Last& last, int mat, int64_t row, int64_t col, bool mirror, float (&v)[32]) {
    if constexpr (C::EP == kNsLast) {
        if (row >= ep.rows) return;
        const int n = ep.cols - col >= 32 ? 32 : int(ep.cols - col);
        const int64_t ld = last.ld[mat];
        if (last.tall >> mat & 1) {             // lanes are neighbours along the result's rows
            const int64_t at = col * ld + row;
            if (last.bf16) {
                uint16_t* const p = static_cast<uint16_t*>(last.p[mat]) + at;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < n) p[c * ld] = to_bf16(v[c] * ep.alpha);
            } else {
                float* const p = static_cast<float*>(last.p[mat]) + at;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < n) p[c * ld] = v[c] * ep.alpha;
            }
            return;
        }
        const int64_t at = row * ld + col;
        if (last.bf16) {
            uint16_t* const p = static_cast<uint16_t*>(last.p[mat]) + at;
            if (n == 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    stu4(p + 8 * g, make_uint4(pack_bf16x2(v[8 * g] * ep.alpha, v[8 * g + 1] * ep.alpha),
                                               pack_bf16x2(v[8 * g + 2] * ep.alpha, v[8 * g + 3] * ep.alpha),
                                               pack_bf16x2(v[8 * g + 4] * ep.alpha, v[8 * g + 5] * ep.alpha),
                                               pack_bf16x2(v[8 * g + 6] * ep.alpha, v[8 * g + 7] * ep.alpha)));
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < n) p[c] = to_bf16(v[c] * ep.alpha);
            }
        } else {
            float* const p = static_cast<float*>(last.p[mat]) + at;
            if (n == 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    st4(p + 4 * g, make_float4(v[4 * g] * ep.alpha, v[4 * g + 1] * ep.alpha, v[4 * g + 2] * ep.alpha, v[4 * g + 3] * ep.alpha));
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < n) p[c] = v[c] * ep.alpha;
            }
        }
    } else {
        const int64_t base = 2 * int64_t(mat) * ep.plane, at = base + row * ep.ldo + col;
        uint32_t hi[16], lo[16];
        if constexpr (C::EP == kNsPoly) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint4 h = ldu4(ep.in + at + 8 * g), l = ldu4(ep.in + at + ep.plane + 8 * g);
                hi[4 * g] = h.x; hi[4 * g + 1] = h.y; hi[4 * g + 2] = h.z; hi[4 * g + 3] = h.w;
                lo[4 * g] = l.x; lo[4 * g + 1] = l.y; lo[4 * g + 2] = l.z; lo[4 * g + 3] = l.w;
            }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            float a = v[2 * c] * ep.alpha, b = v[2 * c + 1] * ep.alpha;
            if constexpr (C::EP == kNsPoly) {
                const float2 f = join2(hi[c], lo[c]);
                a = __fmaf_rn(f.x, ep.beta, a);
                b = __fmaf_rn(f.y, ep.beta, b);
                if (row == col + 2 * c) a += ep.diag;
                if (row == col + 2 * c + 1) b += ep.diag;
            }
            split2(a, b, hi[c], lo[c]);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            stu4(ep.out + at + 8 * g, make_uint4(hi[4 * g], hi[4 * g + 1], hi[4 * g + 2], hi[4 * g + 3]));
            stu4(ep.out + at + ep.plane + 8 * g, make_uint4(lo[4 * g], lo[4 * g + 1], lo[4 * g + 2], lo[4 * g + 3]));
        }
        if (C::TRI && mirror) {
            uint16_t* const p = ep.out + base + col * ep.ldo + row;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                p[c * ep.ldo] = uint16_t(c & 1 ? hi[c / 2] >> 16 : hi[c / 2]);
                p[c * ep.ldo + ep.plane] = uint16_t(c & 1 ? lo[c / 2] >> 16 : lo[c / 2]);
            }
        }
    }
}

template <class C, class Last>
__global__ void __launch_bounds__(kNsThreads, 1)
k_ns(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const NsShape sh,
     const __grid_constant__ NsEpi ep, const __grid_constant__ Last last, uint64_t wait_ns) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = (C::CG == 2 || C::SPLIT) ? cluster_rank() : 0;
    float* const join = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
    const uint32_t bars = smem_addr(smem + C::STAGES * C::STAGE + C::JOIN);
    const uint32_t full = bars, empty = bars + 8 * kNsMaxStages, acc_full = empty + 8 * kNsMaxStages, acc_empty = acc_full + 16,
                   tmem_word = acc_empty + 16, low_empty = bars + 256;
    static_assert(8 * (2 * kNsMaxStages + 5) <= 256, "barriers");
    const bool leader = C::CG == 1 || rank == 0;

    if (warp == 0) tmem_alloc<C::CG>(tmem_word, C::TMEM);
    if (tid == kNsEpiWarps * 32) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
            mbar_init(low_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kNsEpiWarps * C::CG);
        }
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (C::CG == 2 || C::SPLIT) {      // every CTA's barriers exist before any is signalled
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared::cta.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_word) : "memory");
    pdl_wait();
    pdl_trigger();                               // replayed from a graph: 256 x 1024 102 -> 98 us, 8 of them 137 -> 133, Muon's 4 of 777 x 1001 324 -> 317

    const int n_tiles = sh.per * sh.batch;
    const int n_items = C::CUT ? 2 * n_tiles - sh.whole : n_tiles;
    const int n_clusters = C::CG == 2 ? gridDim.x / 2 : C::SPLIT ? gridDim.x / sh.splits : gridDim.x;
    const int cluster = C::CG == 2 ? blockIdx.x / 2 : C::SPLIT ? blockIdx.x / sh.splits : blockIdx.x;
    const int parts = C::SPLIT ? sh.splits : 1;
    const int kb0 = C::SPLIT ? int(int64_t(sh.n_kb) * rank / parts) : 0;
    const int kb1 = C::SPLIT ? int(int64_t(sh.n_kb) * (rank + 1) / parts) : sh.n_kb;

    // Work item w: a matrix, its tile, and whether that is whole (cut 1) or which half of it (cut 2).
    struct Item {
        int mat, mt, nt, sub, cut;
    };
    auto item_at = [&](int w) {
        Item it;
        it.cut = C::CUT && w >= sh.whole ? 2 : 1;
        it.sub = it.cut == 2 ? (w - sh.whole) & 1 : 0;
        const int g = it.cut == 2 ? sh.whole + (w - sh.whole) / 2 : w;
        it.mat = g / sh.per;
        const int t = g - it.mat * sh.per;
        if constexpr (C::TRI) {                  // row mt of tiles has R (mt + 1) of them
            int i = int((sqrtf(8.f * float(t) / float(C::R) + 1.f) - 1.f) * 0.5f);
            while (i > 0 && C::R * i * (i + 1) / 2 > t) --i;
            while (C::R * (i + 1) * (i + 2) / 2 <= t) ++i;
            it.mt = i;
            it.nt = t - C::R * i * (i + 1) / 2;
        } else {                                 // bands of 8 along M: running tiles share operand rows in L2
            const int band = 8 * sh.n_tiles, b = t / band, first = b * 8;
            const int high = sh.m_tiles - first < 8 ? sh.m_tiles - first : 8;
            const int r = t - b * band;
            it.mt = first + r % high;
            it.nt = r / high;
        }
        return it;
    };

    // The pairs' epilogue warpgroups hold 128 sums a thread beside 32 values on their way: they take
    // registers that the third does not need (the launch has 168 per thread of three warpgroups,
    // which ns_launch and the build check; 2 x 208 + 88 = 3 x 168).
    if (warp >= kNsEpiWarps) {
        if constexpr (C::REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kNsEpiWarps) {
            // ---- loads ----
            bool ok = true;
            uint32_t it = 0;
            for (int t = cluster; ok && t < n_items; t += n_clusters) {
                const Item w = item_at(t);
                const int brows = C::BROWS / w.cut;
                const int m0 = (w.mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128;
                const int n0 = w.nt * C::BN + w.sub * (C::BN / w.cut) + (C::CG == 2 ? int(rank) * brows : 0);
                const uint32_t bytes = C::CG * 2 * (C::A_BYTES + C::B_BYTES / w.cut);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % C::STAGES, use = it / C::STAGES;
                    const uint32_t bar = C::CG == 2 ? map_rank(full + 8 * s, 0) : full + 8 * s;
                    const uint32_t st = smem_addr(smem + s * C::STAGE);
#pragma unroll
                    for (int p = 1; p >= 0; --p) {                   // the low planes are free first
                        if (use > 0 && !mbar_wait_bounded((p ? low_empty : empty) + 8 * s, (use - 1) & 1, wait_ns)) {
                            ok = false;
                            break;
                        }
                        if (elect_one()) {
                            if (leader && p == 1) mbar_arrive_tx(full + 8 * s, bytes);
                            const int z = 2 * w.mat + p;
                            const uint32_t a = st + p * C::A_BYTES, b = st + 2 * C::A_BYTES + p * C::B_BYTES;
                            tma_load<C::CG>(a, &map_a, kb * 64, m0, z, bar);
                            tma_load<C::CG>(a + 8192, &map_a, kb * 64, m0 + 64, z, bar);
#pragma unroll
                            for (int c = 0; c < C::BROWS / 64; ++c) {
                                if (c * 64 >= brows) break;
                                if constexpr (C::B_MN) tma_load<C::CG>(b + c * 8192, &map_b, n0 + c * 64, kb * 64, z, bar);
                                else tma_load<C::CG>(b + c * 8192, &map_b, kb * 64, n0 + c * 64, z, bar);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
            }
            // the last use of every stage: its MMAs are done (and, in a pair, their arrivals on this
            // CTA have landed) before the CTA may leave
            for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; ok && k < it; ++k)
                ok = mbar_wait_bounded(empty + 8 * (k % C::STAGES), (k / C::STAGES) & 1, wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) atomicOr(&g_wait_error, 1u);
                const uint64_t t0 = global_ns();                     // copies in flight land within this
                for (int i = 0; i < (1 << 20) && global_ns() - t0 < 2000000ull; ++i) __nanosleep(1000);
            }
            __syncwarp();
        } else if (warp == kNsEpiWarps + 1) {
            // ---- products ----
            if (leader) {
                constexpr uint32_t a_step = 32 / 16, b_step = C::B_MN ? 2048 / 16 : 32 / 16;     // 16 K elements on
                // fp16 operands: the type fields that mma_idesc sets for bf16 cleared
                constexpr uint32_t f16 = ~((1u << 7) | (1u << 10));
                const uint64_t da0 = smem_desc(smem_addr(smem), 16, 1024);
                const uint64_t db0 = smem_desc(smem_addr(smem) + 2 * C::A_BYTES, C::B_MN ? 8192 : 16, 1024);
                bool ok = true;
                uint32_t it = 0;
                for (int t = cluster; ok && t < n_items; t += n_clusters) {
                    const uint32_t idesc = f16 & (C::CUT && t >= sh.whole ? mma_idesc(C::TM, C::BN / 2, false, C::B_MN)
                                                                          : mma_idesc(C::TM, C::BN, false, C::B_MN));
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const uint32_t buf = it & 1, use = it >> 1, s = it % C::STAGES;
                        if (use > 0 && !mbar_wait_bounded(acc_empty + 8 * buf, (use - 1) & 1, wait_ns)) {
                            ok = false;
                            break;
                        }
                        if (!mbar_wait_bounded(full + 8 * s, (it / C::STAGES) & 1, wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + buf * C::BN;
                        const uint64_t das = da0 + s * (C::STAGE / 16), dbs = db0 + s * (C::STAGE / 16);
                        if (elect_one()) {
#pragma unroll
                            for (int pr = 0; pr < 3; ++pr) {         // lo hi, hi lo, hi hi
                                const int pa = pr == 0, pb = pr == 1;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16<C::CG>(d, das + pa * (C::A_BYTES / 16) + k * a_step, dbs + pb * (C::B_BYTES / 16) + k * b_step,
                                                    idesc, pr > 0 || k > 0);
                                if (pr == 1) mma_commit<C::CG>(low_empty + 8 * s);   // its planes can be loaded again
                            }
                            mma_commit<C::CG>(empty + 8 * s);
                            mma_commit<C::CG>(acc_full + 8 * buf);
                        }
                        __syncwarp();
                    }
                }
                if (!__all_sync(0xffffffffu, ok) && lane == 0) atomicOr(&g_wait_error, 1u);
            }
            __syncwarp();
        }
    } else {
        if constexpr (C::REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- sums and epilogue ----
        // Warp w reads TMEM lanes 32 (w mod 4) on, the two halves of the warps alternate groups of 32 columns.
        const int q = warp & 3, half = warp >> 2;
        constexpr int NJ = C::BN / 64;
        bool ok = true;
        uint32_t ac = 0;
        for (int t = cluster; ok && t < n_items; t += n_clusters) {
            const Item w = item_at(t);
            const int nj = w.cut == 2 ? NJ / 2 : NJ;
            float sum[NJ][32];
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[j][i] = 0.f;
            for (int kb = kb0; ok && kb < kb1; ++kb, ++ac) {
                const uint32_t buf = ac & 1;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_full + 8 * buf, (ac >> 1) & 1, wait_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem + buf * C::BN + (uint32_t(q * 32) << 16);
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (j < nj) {
                        float v[32];
                        tmem_ld32(src + (2 * j + half) * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[j][i] += v[i];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (C::CG == 2) mbar_arrive_cluster(map_rank(acc_empty + 8 * buf, 0));
                    else mbar_arrive(acc_empty + 8 * buf);
                }
            }
            if (!ok) break;
            if constexpr (C::SPLIT) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const uint32_t u = 4 * (2 * j + half) + q;   // unit u joins in CTA u mod splits
                    const uint32_t slot = (u / sh.splits) * sh.splits + rank;
                    const uint32_t dst = map_rank(smem_addr(join + slot * kUnitFloats + lane * kUnitLd), u % sh.splits);
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        st_cluster4(dst + 16 * g, sum[j][4 * g], sum[j][4 * g + 1], sum[j][4 * g + 2], sum[j][4 * g + 3]);
                }
            } else {
                const int64_t row = int64_t(w.mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128 + q * 32 + lane;
                const int64_t n0 = int64_t(w.nt) * C::BN + w.sub * (C::BN / w.cut);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    if (j < nj) ns_emit<C>(ep, last, w.mat, row, n0 + (2 * j + half) * 32, w.nt / C::R < w.mt, sum[j]);
            }
        }
        if (!ok && lane == 0) atomicOr(&g_wait_error, 1u);
    }

    // ---- join and teardown: every thread of the cluster gets here ----
    if constexpr (C::SPLIT) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp < kNsEpiWarps) {
            const Item w = item_at(cluster);
            for (int u = int(rank) + warp * sh.splits; u < C::BN / 8; u += kNsEpiWarps * sh.splits) {
                const float* const unit = join + (u / sh.splits) * sh.splits * kUnitFloats + lane * kUnitLd;
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
                for (int r = 0; r < sh.splits; ++r) {
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        const float4 x = ld4(unit + r * kUnitFloats + 4 * g);
                        v[4 * g] += x.x; v[4 * g + 1] += x.y; v[4 * g + 2] += x.z; v[4 * g + 3] += x.w;
                    }
                }
                ns_emit<C>(ep, last, w.mat, int64_t(w.mt) * 128 + (u & 3) * 32 + lane, int64_t(w.nt) * C::BN + (u >> 2) * 32,
                           w.nt / C::R < w.mt, v);
            }
        }
    }
    tc_fence_before();
    if constexpr (C::CG == 2) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc<C::CG>(tmem, C::TMEM);
    }
}

// ---- launches -------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeTiled ns_encode() {
    static std::atomic<EncodeTiled> fn{nullptr};
    EncodeTiled f = fn.load(std::memory_order_relaxed);
    if (!f) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<EncodeTiled>(p);
            fn.store(f, std::memory_order_relaxed);
        }
    }
    return f;
}

// Boxes of 64 columns (128 bytes, 128-byte swizzle) x 64 rows of one plane serve every operand.
cudaError_t ns_map(CUtensorMap* m, const NsPlanes& o, int batch) {
    const EncodeTiled enc = ns_encode();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {cuuint64_t(o.cols), cuuint64_t(o.rows), cuuint64_t(2 * batch)};
    const cuuint64_t strides[2] = {cuuint64_t(o.ld) * 2, cuuint64_t(o.plane) * 2};
    const cuuint32_t box[3] = {64, 64, 1}, ones[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, o.p, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int ns_sms(int dev) {
    static std::atomic<int> n[64];
    if (dev < 0 || dev >= 64) return 0;
    int v = n[dev].load(std::memory_order_relaxed);
    if (v == 0 && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) n[dev].store(v, std::memory_order_relaxed);
    return v;
}

std::atomic<bool> g_ns_launched{false};

cudaError_t take_ns_wait_error(unsigned int* flag) {
    *flag = 0;
    return g_ns_launched.load(std::memory_order_relaxed) ? take_local_wait_error(flag) : cudaSuccess;
}

inline int64_t ns_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class C>
int64_t ns_tiles(const NsProduct& p, int64_t* mt, int64_t* nt) {
    *mt = ns_ceil(p.x.rows, C::TM);
    *nt = ns_ceil(C::TRI ? p.x.rows : p.y.cols, C::BN);
    return C::TRI ? C::R * *mt * (*mt + 1) / 2 - (C::R * *mt - *nt) : *mt * *nt;
}

// Tiles that stay whole: all, or all but those of a last wave at most half full.
template <class C>
int64_t ns_whole(int64_t tiles, int64_t room) {
    const int64_t rem = room > 0 ? tiles % room : 0;
    return C::CUT && 2 * rem <= room ? tiles - rem : tiles;
}

template <class C>
cudaError_t ns_launch(const NsProduct& p, int splits, int dev, cudaStream_t st) {
    using Last = typename std::conditional<C::EP == kNsLast, NsMatrices, NsNoLast>::type;
    static std::atomic<uint64_t> prepared{0};
    cudaError_t e = cudaSuccess;
    if (dev >= 64 || !(prepared.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(k_ns<C, Last>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        cudaFuncAttributes attr;
        if (C::REGS && e == cudaSuccess && (e = cudaFuncGetAttributes(&attr, k_ns<C, Last>)) == cudaSuccess && attr.numRegs != 168)
            e = cudaErrorInvalidConfiguration;
        if (e != cudaSuccess) return e;
        if (dev < 64) prepared.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    CUtensorMap ma, mb;
    if ((e = ns_map(&ma, p.x, p.batch)) != cudaSuccess) return e;
    if ((e = ns_map(&mb, C::EP == kNsGram || C::EP == kNsPoly ? p.x : p.y, p.batch)) != cudaSuccess) return e;
    int64_t mt, nt;
    const int64_t per = ns_tiles<C>(p, &mt, &nt), tiles = per * p.batch, kb = ns_ceil(p.x.cols, 64);
    const int each = C::CG == 2 ? 2 : C::SPLIT ? splits : 1;
    if (tiles * each > INT32_MAX / 16 || kb > INT32_MAX / 128) return cudaErrorInvalidValue;
    const int64_t room = ns_sms(dev) / each, whole = ns_whole<C>(tiles, room);
    const NsShape sh{int32_t(mt), int32_t(nt), int32_t(kb), splits, int32_t(per), p.batch, int32_t(whole)};
    NsEpi ep{p.out.p, p.out.ld, p.out.plane, p.x.p, p.alpha, p.beta, p.diag, int32_t(p.x.rows), int32_t(C::TRI ? p.x.rows : p.y.cols)};
    int64_t clusters = 2 * tiles - whole;
    if (!C::SPLIT && clusters > room) clusters = room > 0 ? room : 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(each);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(clusters * each));
    cfg.blockDim = dim3(kNsThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = each > 1 ? 2 : 1;
    g_ns_launched.store(true, std::memory_order_relaxed);
    Last last{};
    if constexpr (C::EP == kNsLast) last = *p.last;
    return cudaLaunchKernelEx(&cfg, k_ns<C, Last>, ma, mb, sh, ep, last, detail::kWaitNs);
}

// Estimates in us: `fixed` for a launch, `kb` for a K step of 64, `epi` for a tile's stores.
template <class C>
float ns_estimate(const NsProduct& p, int splits, int dev, float fixed, float kb, float epi) {
    int64_t mt, nt;
    const int64_t tiles = ns_tiles<C>(p, &mt, &nt) * p.batch, steps = ns_ceil(p.x.cols, 64);
    if (splits > steps) return 1e30f;
    // clusters of more than two CTAs do not fill every SM
    const int64_t room = C::SPLIT && splits > 2 ? ns_sms(dev) * 9 / 10 / splits : ns_sms(dev) / (C::CG * splits);
    if (room < 1) return 1e30f;
    if (C::SPLIT) return float(ns_ceil(tiles, room)) * (fixed + (splits > 1 ? 0.7f : 0.f) + float(ns_ceil(steps, splits)) * kb + epi);
    const bool cut = ns_whole<C>(tiles, room) < tiles;
    const float waves = float(tiles / room) + (cut ? 0.66f : tiles % room ? 1.f : 0.f);
    return fixed + waves * float(steps) * kb + (cut ? 0.5f : 1.f) * epi;
}

// The configuration with the lowest estimate: 256 or 128 columns of a pair, or 64 of one CTA with
// K over `splits` of them.
struct NsChoice {
    float cost;
    int which, splits;
};
template <int EP>
NsChoice ns_choose(const NsProduct& p, int dev) {
    NsChoice best{ns_estimate<NsCfg<EP, 2, 256, false>>(p, 1, dev, 5.0f, 0.82f, 3.5f), 256, 1};
    auto consider = [&](float cost, int which, int splits) {
        if (cost < best.cost) best = NsChoice{cost, which, splits};
    };
    consider(ns_estimate<NsCfg<EP, 2, 128, false>>(p, 1, dev, 4.0f, 0.46f, 2.5f), 128, 1);
    for (int s = 1; s <= 8; s *= 2) consider(ns_estimate<NsCfg<EP, 1, 64, true>>(p, s, dev, 4.0f, 0.36f, 1.0f), 64, s);
    return best;
}

template <int EP>
float ns_cost(const NsProduct& p) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? ns_choose<EP>(p, dev).cost : 0.f;
}

template <int EP>
cudaError_t ns_product(const NsProduct& p, cudaStream_t st) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const NsChoice c = ns_choose<EP>(p, dev);
    if (c.which == 256) return ns_launch<NsCfg<EP, 2, 256, false>>(p, 1, dev, st);
    if (c.which == 128) return ns_launch<NsCfg<EP, 2, 128, false>>(p, 1, dev, st);
    return ns_launch<NsCfg<EP, 1, 64, true>>(p, c.splits, dev, st);
}

}  // namespace
}  // namespace fsdp
