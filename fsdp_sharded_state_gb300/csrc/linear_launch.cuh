// linear_launch.cuh -- tensor maps, the choice of a configuration and the launches of
// linear_kernel.cuh (host code).
#pragma once

#include "linear_kernel.cuh"

namespace fsdp {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeTiled encode_tiled() {
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

// The map of an operand: boxes of 64 columns (128 bytes, 128-byte swizzle) x box_rows rows
// of one plane; what lies outside the matrix reads as 0.
cudaError_t make_map(CUtensorMap* m, const LinOperand& o, int planes, int box_rows) {
    const EncodeTiled enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {cuuint64_t(o.cols), cuuint64_t(o.rows), cuuint64_t(planes)};
    const cuuint64_t strides[2] = {cuuint64_t(o.ld) * 2, cuuint64_t(planes > 1 ? o.plane : o.ld) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1}, ones[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.ptr), dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int sm_count(int dev) {
    static std::atomic<int> n[64];
    if (dev < 0 || dev >= 64) return 0;
    int v = n[dev].load(std::memory_order_relaxed);
    if (v == 0 && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
        n[dev].store(v, std::memory_order_relaxed);
    return v;
}

// Shared-memory attribute of a kernel, set once per device.
template <class C>
cudaError_t prepare_kernel(int dev) {
    static std::atomic<uint64_t> done{0};
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(k_linear<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (C::REGS && e == cudaSuccess) {             // the registers that the warpgroups share out are there (build.py checks them too)
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, k_linear<C>);
        if (e == cudaSuccess && a.numRegs != 168) return cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How many tiles of a 256-column pair configuration stay whole: all, or all but those of a
// last wave that is at most half full.  Those run in halves: a half's K step takes two thirds
// of a whole tile's (as the 256 x 128 tile's does; quarters took no less), the last wave is
// that much shorter, and so is its epilogue.  4000 x 4000 x 4000 with GELU, dropout and residual:
// 93 us uncut, 88 with 28 of 256 tiles halved.
template <class C>
int64_t whole_tiles(int64_t tiles, int64_t room) {
    const int64_t rem = room > 0 ? tiles % room : 0;
    return C::CUT && 2 * rem <= room ? tiles - rem : tiles;
}

// Whether this translation unit has launched a product (or captured one, to run at any time
// after): before that fsdp_check_status has nothing to ask of it, and reads no word, 9 us each.
std::atomic<bool> g_launched{false};

cudaError_t take_product_wait_error(unsigned int* flag) {
    *flag = 0;
    return g_launched.load(std::memory_order_relaxed) ? take_local_wait_error(flag) : cudaSuccess;
}

// Launches one configuration: splits CTAs per tile (SPLIT), else a persistent grid.
template <class C>
cudaError_t launch_cfg(const LinProblem& p, int splits, cudaStream_t st, int slabs = 1) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = prepare_kernel<C>(dev)) != cudaSuccess) return e;
    CUtensorMap ma, mb;
    if ((e = make_map(&ma, C::ROWS_M ? p.rows_op : p.cols_op, C::PL, C::A_MN ? kKb : 128)) != cudaSuccess) return e;
    if ((e = make_map(&mb, C::ROWS_M ? p.cols_op : p.rows_op, C::PL, C::B_MN ? kKb : C::BBOX)) != cudaSuccess) return e;
    const int64_t M = C::ROWS_M ? p.epi.rows : p.epi.cols, N = C::ROWS_M ? p.epi.cols : p.epi.rows;
    const int64_t mt = ceil_div(M, 128 * C::CG), nt = ceil_div(N, C::BN), kb = ceil_div(p.K, kKb);
    const int per = C::CG == 2 ? 2 : C::SPLIT ? splits : 1;
    // tile numbers, K steps and tile coordinates are 32-bit
    if (mt * nt * per > INT32_MAX / 16 || kb > INT32_MAX / 128 || M > INT32_MAX - 512 || N > INT32_MAX - 512)
        return cudaErrorInvalidValue;
    const int64_t room = sm_count(dev) / per, tiles = mt * nt;
    const int64_t whole = whole_tiles<C>(tiles, room);
    const LinShape sh{int32_t(mt), int32_t(nt), int32_t(kb), splits, slabs, int32_t(whole)};
    int64_t clusters = (2 * tiles - whole) * slabs;
    if (!C::SPLIT && clusters > room) clusters = room > 0 ? room : 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(per);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(clusters * per));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = per > 1 ? 2 : 1;
    g_launched.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, k_linear<C>, ma, mb, sh, p.epi, detail::kWaitNs);
}

// Clusters of `per` CTAs of a kernel that the device holds at once, queried once.
template <class C>
int max_clusters(int dev, int per) {
    static std::atomic<int> known[64][4];
    const int slot = per == 2 ? 1 : per == 4 ? 2 : 3;
    if (per == 1) return sm_count(dev);
    if (dev < 0 || dev >= 64) return sm_count(dev) / (2 * per);
    int n = known[dev][slot].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (prepare_kernel<C>(dev) != cudaSuccess) return 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(per);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(per));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_linear<C>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = sm_count(dev) / (2 * per);
        if (n < 1) n = 1;
    }
    known[dev][slot].store(n, std::memory_order_relaxed);
    return n;
}

// What a configuration costs, in us, measured on GB300 with the operands in L2 or streaming
// from HBM: `fixed` from launch to the first product and from the last store to the end, `kb`
// per K step of 64, `epi` for a tile's epilogue where nothing runs beside it.
struct LinCost {
    float fixed, kb, epi;
};

// A persistent configuration works through its tiles in waves, the epilogues beside the next
// tile's products; a split one runs a cluster per tile, wave after wave.
template <class C>
float estimate(const LinProblem& p, int splits, int dev, LinCost c) {
    const int64_t M = C::ROWS_M ? p.epi.rows : p.epi.cols, N = C::ROWS_M ? p.epi.cols : p.epi.rows;
    const int64_t tiles = ceil_div(M, 128 * C::CG) * ceil_div(N, C::BN), kb = ceil_div(p.K, kKb);
    if (splits > kb) return 1e30f;
    int64_t room;
    if constexpr (C::SPLIT) room = max_clusters<C>(dev, splits);
    else room = sm_count(dev) / C::CG;
    if (room < 1) return 1e30f;
    if (C::SPLIT)
        return float(ceil_div(tiles, room)) * (c.fixed + (splits > 1 ? 0.7f : 0.f) + float(ceil_div(kb, splits)) * c.kb + c.epi);
    const bool cut = whole_tiles<C>(tiles, room) < tiles;
    const float waves = float(tiles / room) + (cut ? 0.66f : tiles % room ? 1.f : 0.f);
    return c.fixed + waves * float(kb) * c.kb + (cut ? 0.5f : 1.f) * c.epi;
}

// The configuration with the lowest estimate.  Measured on GB300 (us, forward, bf16, rows x in
// x out; 256 x 256 pair / 256 x 128 pair / best split): 8192 x 4096 x 11008 382 / 452 / 1248;
// 2048^3 15.6 / 16.4 / 27; 333 x 2048 x 2048 - / 11 / 11; 1 x 2048 x 2048 13.3 / 9.2 / 5.8 (32
// columns, 4 CTAs per tile), where one CTA per tile takes 9.8 and 8 CTAs, two waves of
// clusters, 9.3.
//
// For bf16 results with aligned rows the pair configurations are compiled for each activation
// and dropout (launch_pair, in a translation unit of its own); the others take them at run
// time: split tiles run their epilogue once, and fp32 tiles have six times the products to run
// it beside.
template <int MODE, typename OT, int PL, int CH>
cudaError_t launch_product(const LinProblem& p, cudaError_t (*launch_pair)(const LinProblem&, int, cudaStream_t), cudaStream_t st) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    using P256 = LinCfg<MODE, OT, 2, 256, PL, CH, false>;
    using P128 = LinCfg<MODE, OT, 2, 128, PL, CH, false>;
    using S128 = LinCfg<MODE, OT, 1, 128, 1, CH, true>;
    using S64 = LinCfg<MODE, OT, 1, 64, PL, CH, true>;
    using S32 = LinCfg<MODE, OT, 1, MODE == kWgrad ? 64 : 32, PL, CH, true>;
    constexpr float f = PL == 1 ? 1.f : 6.f;
    float best = estimate<P256>(p, 1, dev, {5.0f, 0.275f * f, 3.5f});
    int which = 256, splits = 1;
    auto consider = [&](float cost, int w, int s) {
        if (cost < best) {
            best = cost;
            which = w;
            splits = s;
        }
    };
    consider(estimate<P128>(p, 1, dev, {3.9f, PL == 1 ? 0.18f : 1.05f, 2.5f}), 128, 1);
    for (int s = 1; s <= 8; s *= 2) {
        if constexpr (PL == 1) consider(estimate<S128>(p, s, dev, {4.3f, 0.25f, 2.0f}), 2, s);
        consider(estimate<S64>(p, s, dev, {4.2f, PL == 1 ? 0.21f : 0.70f, 1.0f}), 1, s);
        if constexpr (MODE != kWgrad) consider(estimate<S32>(p, s, dev, {4.0f, PL == 1 ? 0.20f : 0.63f, 0.5f}), 0, s);
    }
    if (p.slabs > 1 && best > 4.2f + float(ceil_div(ceil_div(p.K, kKb), kSlabSplits * p.slabs)) * (PL == 1 ? 0.21f : 0.70f) + 4.5f) {
        // a small out and many rows: slabs of K over clusters, and a launch that adds them up
        if constexpr (MODE == kWgrad) return launch_wgrad_slabs(p, st);
    }
    switch (which) {
        case 0:
            if constexpr (MODE != kWgrad) return launch_cfg<S32>(p, splits, st);
            break;
        case 1: return launch_cfg<S64>(p, splits, st);
        case 2:
            if constexpr (PL == 1) return launch_cfg<S128>(p, splits, st);
            break;
        default: return launch_pair(p, which, st);
    }
    return cudaErrorInvalidValue;
}

template <int MODE, typename OT, int PL, int CH, int EP = -1, bool ANY = false>
cudaError_t launch_pair_as(const LinProblem& p, int bn, cudaStream_t st) {
    return bn == 256 ? launch_cfg<LinCfg<MODE, OT, 2, 256, PL, CH, false, EP, ANY>>(p, 1, st)
                     : launch_cfg<LinCfg<MODE, OT, 2, 128, PL, CH, false, EP, ANY>>(p, 1, st);
}

}  // namespace
}  // namespace fsdp
