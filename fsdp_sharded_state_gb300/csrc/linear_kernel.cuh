// linear_kernel.cuh -- the matrix kernel of the linear layers (sm_103a).
//
// D[M, N] = sum over k of A[M, k] B[N, k] on the 5th-generation tensor cores, fp32
// accumulators in TMEM, with the layer's epilogue (linear_epilogue.cuh) applied before the one
// rounding to the output type.
//
// Roles of a CTA (12 warps): warp 8 loads the operand tiles with tensor-map copies into a
// ring of stages, warp 9 issues the MMAs (both with the whole warp in the loop and one elected
// lane issuing: with the loop inside one lane's branch each MMA cost some 100 clocks to issue,
// and no configuration did a K step in under 540), warps 0-7 empty the accumulators, and in
// wgrad warps 10 and 11 add up the columns of dz for db.  The accumulators are double-buffered,
// so a persistent CTA's epilogue runs beside the next tile's products.  Operands keep the
// row-major layout that the user's tensors have: the matrix descriptors take K-major tiles
// (forward: w and x; dgrad: dz) and MN-major tiles (dgrad: w; wgrad: dz and x), so nothing is
// transposed in memory.
//
// What bounds it.  A CTA alone reads 12 KB of shared memory per MMA of 128 x 256 x 16 and 128
// clocks and has as much written by the copies: 192 bytes a clock where 128 go through.  A pair
// of CTAs (cta_group::2) shares the B operand: 64 + 64 bytes a clock per SM, and 512 clocks per
// K step of 64.  Measured on GB300, bf16: the bare product 8192 x 4096 x 11008, the same call in
// a short loop, 377-402 us, 1.84-1.96 PFLOP/s (the library's burst is 1.87, its sustained rate 1.73);
// with the epilogues of training, other work in between, 1.58-1.70; ncu counts the tensor pipe
// active in 93-96 % of cycles.  Against the bare product 128 x 128 tiles of one CTA reach 1.21 and
// pairs with 256 x 128 1.63 PFLOP/s; these and the splits of K over a cluster are for sizes with
// too few 256 x 256 tiles.  Below K of about 2500 a heavy epilogue (dropout and gelu', two matrices
// read) takes longer than its tile's products: see RowsEmit.
//
// fp32 operands come as three bf16 planes: six products per K step, 3072 clocks of MMA on 96 KB
// of stage, so the pairs run at the same rate (4096 x 2048 x 5504: 286 us, 323 TFLOP/s of fp32
// products, 1.94 PFLOP/s of bf16 ones).  The tensor cores round the accumulator towards zero at
// every step: measured 1.6e-8 of the sum per step of 16 products, 9e-6 at K = 8192.  Where the
// result is fp32 the accumulators are therefore emptied into fp32 registers every CH K steps
// (8 for bf16 operands, 2 for fp32 ones with the small products first): relative error 5e-7 and
// 3e-7 at every K, for 8 % of the time at bf16.  bf16 results keep the whole K in the
// accumulators: the loss is far below their rounding.  At 8192 x 11008 -> 4096, 0.6 % of them are not
// the nearest value (a plain fp32 product: 0.06 %), and the error against 64 bits is 1.64521e-3 in
// norm, 1.64517e-3 for the exact results rounded.
//
// Every wait on an mbarrier is bounded; a role that gives up records it (g_wait_error of
// this translation unit, read by fsdp_check_status), lets copies in flight land and goes
// to the teardown, which every thread of the CTA (and of the cluster) reaches on every path.
#pragma once

#include "linear_epilogue.cuh"

namespace fsdp {
namespace {

// A kernel configuration.  CG CTAs share a tile of 128 CG x BN; PL bf16 planes per operand
// (3 planes: six products, of the terms whose exponents add up to at most two steps); CH:
// K steps after which the accumulators are added to fp32 registers (0: never).  SPLIT: the
// CTAs of a cluster (2, 4 or 8, CG = 1) take a share of K each and join through shared memory.
template <int MODE_, typename OT_, int CG_, int BN_, int PL_, int CH_, bool SPLIT_, int EP_ = -1, bool ANY_ = false>
struct LinCfg {
    using OT = OT_;
    static constexpr int MODE = MODE_, CG = CG_, BN = BN_, PL = PL_, CH = CH_, EP = EP_;
    static constexpr bool SPLIT = SPLIT_;
    // Which of out's axes runs along M.  A split tile of forward or dgrad has the features
    // there, so that few rows need few columns of the tile; the others have out's rows, of which
    // a lane then holds consecutive columns (a unit through shared memory took 1,150 clocks,
    // 2,200 with a column per lane).
    static constexpr bool ROWS_M = MODE == kWgrad || !SPLIT;
    static constexpr bool A_MN = MODE == kWgrad || (MODE == kDgrad && !ROWS_M);
    static constexpr bool B_MN = MODE == kWgrad || (MODE == kDgrad && ROWS_M);
    static constexpr bool REGS = !SPLIT;                                    // see setmaxnreg below
    // ANY: rows of the epilogue's matrices start anywhere, else (DIRECT) they are aligned to 32
    // bytes; kernels of their own, since one with both forms was 6 % slower for its code's size.
    static constexpr bool ANY = ANY_;
    static constexpr bool DIRECT = !SPLIT && CH == 0 && sizeof(OT) == 2;    // RowsEmit where rows are aligned
    static constexpr int BROWS = BN / CG;                        // B rows a CTA loads
    static constexpr bool CUT = CG == 2 && BN == 256;            // tiles of the last wave may be halved
    static constexpr int BBOX = CUT ? BROWS / 2 : BROWS;         // rows of a K-major copy: half a tile's, or all
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BROWS * 128;
    static constexpr int STAGE = PL * (A_BYTES + B_BYTES);
    // the epilogue's shared memory: a unit per warp, or the join's slots
    static constexpr int EPI = SPLIT ? (BN >= 128 ? 64 : 32) * 1024 : kEpiWarps * kUnitFloats * 4;
    static constexpr int MORE = 2048;                       // alignment, barriers, column sums
    static constexpr int FIT = (227 * 1024 - MORE - EPI) / STAGE;
    static constexpr int STAGES = FIT < kLinMaxStages ? FIT : kLinMaxStages;
    static constexpr int SMEM = STAGES * STAGE + EPI + MORE;
    static constexpr int TMEM = 2 * BN < 32 ? 32 : 2 * BN;
    static_assert(STAGES >= 2, "two stages");
    static_assert(SMEM > 114 * 1024 && SMEM <= 227 * 1024, "one CTA per SM: its TMEM is never contended");
    static_assert(!B_MN || BROWS % 64 == 0, "MN-major tiles come in chunks of 64");
    static_assert(!SPLIT || CG == 1, "a cluster is a pair or a split");
};

// splits: CTAs per tile; slabs (wgrad): K ranges with an output of their own each, [slabs][rows][ldo].
// The work of the 256-column pairs: the first `whole` tiles as they are, the others, less than
// half a wave, in halves of 128 columns, so that the last wave is spread over the pairs.
struct LinShape {
    int32_t m_tiles, n_tiles, n_kb, splits, slabs, whole;
};

// The two warps that add dz up, and no others.
__device__ __forceinline__ void sum_warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kSumWarps) : "memory"); }

template <class C>
__global__ void __launch_bounds__(kLinThreads, 1)
k_linear(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const LinShape sh,
         const __grid_constant__ LinEpi ep, uint64_t wait_ns) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = (C::CG == 2 || C::SPLIT) ? cluster_rank() : 0;
    float* const epi_smem = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
    const uint32_t bars = smem_addr(smem + C::STAGES * C::STAGE + C::EPI);
    const uint32_t full = bars, empty = bars + 8 * kLinMaxStages, acc_full = empty + 8 * kLinMaxStages,
                   acc_empty = acc_full + 16, tmem_word = acc_empty + 16;
    static_assert(8 * (2 * kLinMaxStages + 5) <= 256, "barriers");
    float* const db_part = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE + C::EPI + 256);   // [128]
    // a stage's plane may be loaded again: plane 0 with the stage, planes 1 and 2 earlier
    auto plane_empty = [&](int p) { return p == 0 ? empty : bars + 768 + 8 * kLinMaxStages * (p - 1); };
    const bool leader = C::CG == 1 || rank == 0;

    if (warp == 0) tmem_alloc<C::CG>(tmem_word, C::TMEM);
    if (tid == kEpiWarps * 32) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            for (int p = 0; p < C::PL; ++p) mbar_init(plane_empty(p) + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kEpiWarps * C::CG);
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

    const int n_tiles = sh.m_tiles * sh.n_tiles;
    const int n_clusters = C::CG == 2 ? gridDim.x / 2 : C::SPLIT ? gridDim.x / sh.splits : gridDim.x;
    const int slab = C::SPLIT && C::MODE == kWgrad ? blockIdx.x / sh.splits / n_tiles : 0;
    const int cluster = C::CG == 2 ? blockIdx.x / 2 : C::SPLIT ? blockIdx.x / sh.splits - slab * n_tiles : blockIdx.x;
    // this CTA's K steps
    const int parts = C::SPLIT ? sh.splits * sh.slabs : 1, part = C::SPLIT ? slab * sh.splits + int(rank) : 0;
    const int kb0 = C::SPLIT ? int(int64_t(sh.n_kb) * part / parts) : 0;
    const int kb1 = C::SPLIT ? int(int64_t(sh.n_kb) * (part + 1) / parts) : sh.n_kb;
    const int chunk = C::CH ? C::CH : sh.n_kb;

    // Who adds dz up (wgrad's db): so many tiles of a row of tiles, so many columns each.
    const int db_tiles = sh.n_tiles >= 8 ? 8 : sh.n_tiles >= 4 ? 4 : sh.n_tiles >= 2 ? 2 : 1;
    const int db_width = ep.rows > 64 ? 128 : ep.rows > 32 ? 64 : 32;
    const int db_cols = db_width / db_tiles > 16 ? db_width / db_tiles : 16;

    // Tiles in bands of 8 along M, N outer inside a band: concurrently running tiles share
    // operand rows in L2.
    auto tile_at = [&](int t, int& mt, int& nt) {
        const int band = 8 * sh.n_tiles, g = t / band, first = g * 8;
        const int high = sh.m_tiles - first < 8 ? sh.m_tiles - first : 8;
        const int r = t - g * band;
        mt = first + r % high;
        nt = r / high;
    };
    // Work item w: its tile, and whether that is whole (cut 1) or which half of it (cut 2).
    const int n_items = C::CUT ? 2 * n_tiles - sh.whole : n_tiles;
    struct Item {
        int mt, nt, sub, cut;
    };
    auto item_at = [&](int w) {
        Item it;
        it.cut = C::CUT && w >= sh.whole ? 2 : 1;
        it.sub = it.cut == 2 ? (w - sh.whole) & 1 : 0;
        tile_at(it.cut == 2 ? sh.whole + (w - sh.whole) / 2 : w, it.mt, it.nt);
        return it;
    };

    // Kernels that hold sums in registers: the epilogue's two warpgroups take registers that the
    // third does not need (the launch has 168 per thread of three warpgroups, which prepare_kernel
    // checks; 2 x 208 + 88 = 2 x 200 + 104 = 3 x 168).  Spilled, the sums went through an L1 of the 28 KB that shared memory leaves, and a
    // chunk of 128 columns took a warp 6,000 clocks to add instead of 2,000.
    if (warp >= kEpiWarps) {
        if constexpr (C::REGS && C::MODE == kWgrad) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        else if constexpr (C::REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == kEpiWarps) {
            // ---- loads ----
            bool ok = true;
            uint32_t it = 0;
            for (int t = cluster; ok && t < n_items; t += n_clusters) {
                const Item w = item_at(t);
                const int nt = w.nt, brows = C::BROWS / w.cut;
                const int m0 = (w.mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128;
                const int n0 = nt * C::BN + w.sub * (C::BN / w.cut) + (C::CG == 2 ? int(rank) * brows : 0);
                constexpr int BBOX_BYTES = C::B_MN ? 8192 : C::BBOX * 128;
                const int bboxes = C::B_BYTES / BBOX_BYTES / w.cut;
                const uint32_t bytes = C::CG * C::PL * (C::A_BYTES + C::B_BYTES / w.cut);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % C::STAGES, use = it / C::STAGES;
                    const uint32_t bar = C::CG == 2 ? map_rank(full + 8 * s, 0) : full + 8 * s;
                    const uint32_t st = smem_addr(smem + s * C::STAGE);
#pragma unroll
                    for (int p = C::PL - 1; p >= 0; --p) {           // in the order in which the products free the planes
                        if (use > 0 && !mbar_wait_bounded(plane_empty(p) + 8 * s, (use - 1) & 1, wait_ns)) {
                            ok = false;
                            break;
                        }
                        if (elect_one()) {
                            if (leader && p == C::PL - 1) mbar_arrive_tx(full + 8 * s, bytes);
                            const uint32_t a = st + p * C::A_BYTES, b = st + C::PL * C::A_BYTES + p * C::B_BYTES;
                            if constexpr (C::A_MN) {
                                tma_load<C::CG>(a, &map_a, m0, kb * kKb, p, bar);
                                tma_load<C::CG>(a + 8192, &map_a, m0 + 64, kb * kKb, p, bar);
                            } else {
                                tma_load<C::CG>(a, &map_a, kb * kKb, m0, p, bar);
                            }
#pragma unroll
                            for (int c = 0; c < C::B_BYTES / BBOX_BYTES; ++c) {
                                if (c >= bboxes) break;
                                if constexpr (C::B_MN) tma_load<C::CG>(b + c * BBOX_BYTES, &map_b, n0 + c * 64, kb * kKb, p, bar);
                                else tma_load<C::CG>(b + c * BBOX_BYTES, &map_b, kb * kKb, n0 + c * C::BBOX, p, bar);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
            }
            // the last use of every stage: its MMAs are done (and, in a pair, their arrivals on
            // this CTA have landed) before the CTA may leave
            for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; ok && k < it; ++k)
                ok = mbar_wait_bounded(empty + 8 * (k % C::STAGES), (k / C::STAGES) & 1, wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) atomicOr(&g_wait_error, 1u);
                const uint64_t t0 = global_ns();                 // copies in flight land within this
                for (int i = 0; i < (1 << 20) && global_ns() - t0 < 2000000ull; ++i) __nanosleep(1000);
            }
            __syncwarp();
        } else if (warp == kEpiWarps + 1) {
            // ---- products ----
            if (leader) {
                // 16 K elements on: 32 bytes along a K-major row, 16 rows of an MN-major tile
                constexpr uint32_t a_step = C::A_MN ? 2048 / 16 : 32 / 16, b_step = C::B_MN ? 2048 / 16 : 32 / 16;
                const uint64_t da0 = smem_desc(smem_addr(smem), C::A_MN ? 8192 : 16, 1024);
                const uint64_t db0 = smem_desc(smem_addr(smem) + C::PL * C::A_BYTES, C::B_MN ? 8192 : 16, 1024);
                bool ok = true;
                uint32_t it = 0, ac = 0;
                for (int t = cluster; ok && t < n_items; t += n_clusters) {
                    const uint32_t idesc = C::CUT && t >= sh.whole ? mma_idesc(128 * C::CG, C::BN / 2, C::A_MN, C::B_MN)
                                                                   : mma_idesc(128 * C::CG, C::BN, C::A_MN, C::B_MN);
                    for (int kc = kb0; ok && kc < kb1; kc += chunk, ++ac) {
                        const uint32_t buf = ac & 1, use = ac >> 1;
                        if (use > 0 && !mbar_wait_bounded(acc_empty + 8 * buf, (use - 1) & 1, wait_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + buf * C::BN;
                        const int ke = kc + chunk < kb1 ? kc + chunk : kb1;
                        for (int kb = kc; kb < ke; ++kb, ++it) {
                            const uint32_t s = it % C::STAGES;
                            if (!mbar_wait_bounded(full + 8 * s, (it / C::STAGES) & 1, wait_ns)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            // stages are far below the descriptor's 256 KB, so offsets add to its low bits
                            const uint64_t das = da0 + s * (C::STAGE / 16), dbs = db0 + s * (C::STAGE / 16);
                            if (elect_one()) {
#pragma unroll
                                for (int pr = 0; pr < (C::PL == 3 ? 6 : 1); ++pr) {
                                    // plane pairs (0,2) (2,0) (1,1) (0,1) (1,0) (0,0), smallest first (the other
                                    // three are below 2^-24 of the product)
                                    const int pa = C::PL == 1 ? 0 : pr == 1 ? 2 : pr == 2 || pr == 4 ? 1 : 0;
                                    const int pb = C::PL == 1 ? 0 : pr == 0 ? 2 : pr == 2 || pr == 3 ? 1 : 0;
#pragma unroll
                                    for (int k = 0; k < kKb / 16; ++k)
                                        mma_bf16<C::CG>(d, das + pa * (C::A_BYTES / 16) + k * a_step,
                                                        dbs + pb * (C::B_BYTES / 16) + k * b_step, idesc, kb > kc || pr > 0 || k > 0);
                                    // the low planes are in the first two products alone, the middle ones in the
                                    // next three: their places can be loaded again before the stage is done
                                    if (C::PL == 3 && pr == 1) mma_commit<C::CG>(plane_empty(2) + 8 * s);
                                    if (C::PL == 3 && pr == 4) mma_commit<C::CG>(plane_empty(1) + 8 * s);
                                }
                                mma_commit<C::CG>(empty + 8 * s);
                                if (kb + 1 == ke) mma_commit<C::CG>(acc_full + 8 * buf);
                            }
                            __syncwarp();
                        }
                    }
                }
                if (!__all_sync(0xffffffffu, ok) && lane == 0) atomicOr(&g_wait_error, 1u);
            }
            __syncwarp();
        } else if (warp >= kEpiWarps + 2) {
            // ---- column sums of dz ----
            const int half = warp - (kEpiWarps + 2);
            if constexpr (C::MODE == kWgrad) {
                // the tiles of a row of tiles belong to the same columns of dz: the first db_tiles of
                // them take db_cols each, of the K steps that are this CTA's, half of the rows a warp
                using DT = typename std::conditional<C::PL == 3, float, uint16_t>::type;
                using RS = RowSum<DT>;
                const int lanes = db_cols / RS::E;
                const int64_t row = int64_t(kb0) * kKb, rows = (int64_t(kb1) * kKb < ep.dz_rows ? int64_t(kb1) * kKb : ep.dz_rows) - row;
                for (int t = cluster; ep.db && t < n_items; t += n_clusters) {
                    const Item w = item_at(t);
                    const int64_t col = int64_t(w.mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128 + w.nt * db_cols;
                    if (w.nt >= db_tiles || w.sub > 0 || col >= ep.rows) continue;
                    RS db = {};
                    db.add(static_cast<const DT*>(ep.dz) + row * ep.lddz, ep.lddz, half, rows, col, ep.rows, ep.dz_vec, lanes, lane);
                    db.join(lanes);
                    if (half == 1 && lane < lanes) {
#pragma unroll
                        for (int e = 0; e < RS::E; ++e) db_part[lane * RS::E + e] = db.v[e];
                    }
                    sum_warps_sync();
                    if (half == 0 && lane < lanes) {
#pragma unroll
                        for (int e = 0; e < RS::E; ++e) {
                            const int64_t c = col + lane * RS::E + e;
                            db.v[e] += db_part[lane * RS::E + e];
                            if constexpr (C::SPLIT) db_part[lane * RS::E + e] = db.v[e];
                            else if (c < ep.rows) emit_db<typename C::OT>(ep, c, db.v[e]);
                        }
                    }
                    sum_warps_sync();
                }
            }
            __syncwarp();
        }
    } else {
        if constexpr (C::REGS && C::MODE == kWgrad) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        else if constexpr (C::REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- epilogue ----
        // Warp w reads TMEM lanes 32 (w mod 4) on: rows 32 q of the CTA's part of the tile; the
        // two halves of the warps take alternate groups of 32 columns, so that they write a line of
        // 128 bytes at about the same time; where rows are not aligned (RowsEmit's windows run on
        // from group to group) half of the columns each.
        const int q = warp & 3, half = warp >> 2;
        constexpr int NJ = (C::BN + 63) / 64;                // groups of 32 columns per warp
        bool ok = true;
        uint32_t ac = 0;
        for (int t = cluster; ok && t < n_items; t += n_clusters) {
            const Item w = item_at(t);
            const int nj = NJ / w.cut;                               // of this item
            auto group = [&](int jj) { return C::DIRECT && C::ANY ? half * nj + jj : 2 * jj + half; };
            const int64_t m0 = int64_t(w.mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128 + q * 32;
            const int64_t n0 = int64_t(w.nt) * C::BN + w.sub * (C::BN / w.cut);
            float sum[C::CH ? NJ : 1][32];
            if constexpr (C::CH != 0) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[j][i] = 0.f;
            }
            constexpr bool WHOLE = C::CH != 0 && C::MODE == kWgrad && !C::SPLIT && sizeof(typename C::OT) == 4;
            const bool whole = WHOLE && ep.vec == 2 && w.cut == 1 && n0 + C::BN <= ep.cols;
            if constexpr (WHOLE) {
                if (whole && ep.accumulate) prefetch_sums<NJ>(ep, m0 + lane, n0 + half * 32);
            }
            UnitEmit<C::MODE, typename C::OT, C::EP> io;
            auto begin = [&](int jj) {
                const int64_t n = n0 + group(jj) * 32;
                if constexpr (!C::SPLIT) io.begin(ep, C::ROWS_M ? m0 : n, C::ROWS_M ? n : m0, lane);
            };
            auto finish = [&](int jj, const float (&v)[32]) {
                const int j = group(jj);                     // this group of 32 columns
                if constexpr (C::SPLIT) {
                    const uint32_t u = 4 * j + q;            // unit u joins in CTA u mod splits
                    const uint32_t slot = (u / sh.splits) * sh.splits + rank;
                    const uint32_t dst = map_rank(smem_addr(epi_smem + slot * kUnitFloats), u % sh.splits);
                    if constexpr (C::ROWS_M) {               // a lane holds a row
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            st_cluster4(dst + 4 * unit_at(lane, 4 * g), v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
                    } else {                                 // a lane holds a column
#pragma unroll
                        for (int c = 0; c < 32; ++c) st_cluster(dst + 4 * unit_at(c, lane), v[c]);
                    }
                } else {
                    float* const unit = epi_smem + warp * kUnitFloats;
                    __syncwarp();
                    if constexpr (C::ROWS_M) {               // a lane holds a row
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            st4(unit + unit_at(lane, 4 * g), make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]));
                    } else {                                 // a lane holds a column
#pragma unroll
                        for (int c = 0; c < 32; ++c) unit[unit_at(c, lane)] = v[c];
                    }
                    __syncwarp();
                    io.run(ep, unit, 1, lane);
                }
            };
            for (int kc = kb0; ok && kc < kb1; kc += chunk, ++ac) {
                const uint32_t buf = ac & 1;
                RowsEmit<C::MODE, C::EP, !C::ANY> rows;
                bool direct = C::DIRECT;
                if constexpr (C::DIRECT) rows.begin(ep, m0 + lane, n0 + group(0) * 32, nj);
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_full + 8 * buf, (ac >> 1) & 1, wait_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t src = tmem + buf * C::BN + (uint32_t(q * 32) << 16);
                DropRow dr = {};
                DropCol* const dcol = reinterpret_cast<DropCol*>(epi_smem + warp * kUnitFloats);
                if constexpr (C::DIRECT && C::MODE != kWgrad) {
                    if (direct && (C::EP >= 0 ? C::EP >= 4 : ep.drop.on != 0)) {
                        // the generator's products of the lane's row, and, one block per lane, of this
                        // warp's columns; a batch that crosses 2^32 rows takes the other path
                        const uint64_t r0 = uint64_t(m0 + ep.drop.row0);
                        const uint32_t hi = uint32_t(r0 >> 32);
                        direct = hi == uint32_t((r0 + 31) >> 32);
                        dr = drop_row(ep.drop, uint32_t(r0) + lane, __umulhi(0xCD9E8D57u, hi));
                        __syncwarp();
                        if (lane < NJ * 8)
                            dcol[lane] = drop_col(ep.drop, uint32_t((n0 + group(lane >> 3) * 32) >> 2) + (lane & 7), hi);
                        __syncwarp();
                    }
                }
                int done = 0;                                // units of the direct path
                if constexpr (C::DIRECT) {
                    if (direct) done = m0 >= ep.rows ? NJ : rows.run(ep, src + group(0) * 32, dr, dcol);
                }
                constexpr int kUnrollUnits = C::CH != 0 ? NJ : 1;
#pragma unroll kUnrollUnits
                for (int jj = C::DIRECT ? done : 0; jj < NJ; ++jj) {
                    if (jj < nj && group(jj) * 32 < C::BN) {
                        if constexpr (C::CH != 0) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                Acc16 a;
                                float v[16];
                                tmem_ld16_async(src + group(jj) * 32 + 16 * h, a);
                                tmem_wait_ld16(a, v);
#pragma unroll
                                for (int i = 0; i < 16; ++i) sum[jj][16 * h + i] += v[i];
                            }
                        } else {
                            float v[32];
                            begin(jj);
                            tmem_ld32(src + group(jj) * 32, v);
                            finish(jj, v);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (C::CG == 2) mbar_arrive_cluster(map_rank(acc_empty + 8 * buf, 0));
                    else mbar_arrive(acc_empty + 8 * buf);
                }
            }
            if constexpr (C::CH != 0) {
                if constexpr (WHOLE) {
                    if (ok && whole) emit_sums<NJ>(ep, sum, m0 + lane, n0 + half * 32);
                }
#pragma unroll
                for (int jj = 0; jj < NJ; ++jj)
                    if (ok && !whole && jj < nj && group(jj) * 32 < C::BN) {
                        begin(jj);
                        finish(jj, sum[jj]);
                    }
            }
        }
        if (!ok && lane == 0) atomicOr(&g_wait_error, 1u);
    }

    // ---- join and teardown: every thread of the cluster gets here ----
    if constexpr (C::SPLIT) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp < kEpiWarps) {
            int mt, nt;
            tile_at(cluster, mt, nt);
            for (int u = int(rank) + warp * sh.splits; u < C::BN / 8; u += kEpiWarps * sh.splits) {
                const int q = u & 3, j = u >> 2;
                const int64_t m0 = int64_t(mt) * 128 + q * 32, n0 = int64_t(nt) * C::BN + j * 32;
                UnitEmit<C::MODE, typename C::OT, C::EP> io;
                io.begin(ep, C::ROWS_M ? m0 : n0, C::ROWS_M ? n0 : m0, lane, C::MODE == kWgrad ? slab * ep.rows : 0);
                io.run(ep, epi_smem + (u / sh.splits) * sh.splits * kUnitFloats, sh.splits, lane);
            }
        }
        if constexpr (C::MODE == kWgrad) {
            if (ep.db) {                         // the CTAs' shares of the column sums, in order
                int mt, nt;
                tile_at(cluster, mt, nt);
                const int64_t c = int64_t(mt) * 128 + nt * db_cols + tid;
                if (rank == 0 && nt < db_tiles && tid < db_cols && c < ep.rows) {
                    float t = 0.f;
                    for (int r = 0; r < sh.splits; ++r) t += ld_cluster(map_rank(smem_addr(db_part + tid), r));
                    emit_db<typename C::OT>(ep, c + slab * ep.rows, t);
                }
                __syncwarp();
                cluster_arrive();                // no CTA leaves while its share is read
                cluster_wait();
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

}  // namespace
}  // namespace fsdp
