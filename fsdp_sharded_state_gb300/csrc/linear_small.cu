// linear_small.cu -- fp32 products of small matrices on the FMA units: no splitting into bf16
// terms, whose launch alone takes longer than such a product.
//
// A CTA takes 32 x 32 of out and a range of K in steps of 64: a step's operands lie in shared
// memory as [64 k][32], whichever way they run in memory, and its eight warps take every eighth
// k each, a lane 4 x 8 of out (three 16-byte reads to 32 FMAs); the warps' sums join at the end.
// wgrad's K is its rows: slabs of them get partial sums of their own, added by a second launch.
// Products and sums are fp32; the order of a sum depends on the sizes alone.  Bound by the FMA
// units and, smallest, by latency: a step's operands are fetched while the one before is
// computed, 0.8 us where an SM has one CTA.
#include "linear_launch.cuh"

namespace fsdp {
namespace {

constexpr int kSmThreads = 256, kSmWarps = 8, kSmK = 64, kSmSide = 32, kSmLoads = kSmK * kSmSide / kSmThreads;

// A step of one operand on its way from memory to shared memory.  K_ROWS: k runs along the
// matrix's rows (element (i, k) at p[k * ld + i]), else along its columns.  A warp reads 32 elements of
// a row, or 8 of 4 rows, so that its stores meet 32 banks.
template <bool K_ROWS>
struct SmallStep {
    const float* p;            // this thread's first element of the next step
    int64_t every, step;       // from one of its elements to the next, from step to step
    int in, k, at;             // its elements inside the matrix along the side (K_ROWS: all or none); its first k; place in shared memory
    float v[kSmLoads];

    __device__ __forceinline__ void begin(const float* m, int64_t ld, int64_t i0, int64_t n, int64_t k0) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int i = K_ROWS ? lane : lane >> 3;
        k = K_ROWS ? warp : 8 * warp + (lane & 7);
        at = K_ROWS ? unit_at(warp, lane) : 32 * k;
        p = K_ROWS ? m + (k0 + k) * ld + i0 + i : m + (i0 + i) * ld + k0 + k;
        every = (K_ROWS ? 8 : 4) * ld;
        step = K_ROWS ? kSmK * ld : kSmK;
        const int64_t left = n - i0 - i;                         // K_ROWS: side i alone; else sides i, i + 4, ..
        in = K_ROWS ? left > 0 : left <= 0 ? 0 : left >= kSmSide ? kSmLoads : int(left + 3) >> 2;
    }
    // The next step, of which `left` k are there.
    __device__ __forceinline__ void load(int64_t left) {
        const int l = left < kSmK ? int(left) : kSmK;
        const float* q = p;
#pragma unroll
        for (int j = 0; j < kSmLoads; ++j) {
            v[j] = (K_ROWS ? in && k + 8 * j < l : j < in && k < l) ? *q : 0.f;
            q += every;
        }
        p += step;
    }
    __device__ __forceinline__ void store(float* s) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < kSmLoads; ++j) s[K_ROWS ? at + 8 * 32 * j : at + ((j ^ (lane & 7)) << 2 | lane >> 3)] = v[j];
    }
};

template <int MODE, typename OT>
__global__ void __launch_bounds__(kSmThreads, 2)
k_small(const float* __restrict__ a, int64_t lda, const float* __restrict__ b, int64_t ldb, int64_t K, int64_t slab_k,
        const __grid_constant__ LinEpi ep) {
    __shared__ __align__(16) float sm[kSmWarps * kUnitFloats];   // two steps of both operands; at the end a unit per warp
    __shared__ float sums[kSmWarps][kSmSide];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ly = lane >> 2, lx = lane & 3;
    const int64_t m0 = int64_t(blockIdx.y) * kSmSide, n0 = int64_t(blockIdx.x) * kSmSide;
    const int64_t k0 = blockIdx.z * slab_k, k1 = k0 + slab_k < K ? k0 + slab_k : K;
    SmallStep<MODE == kWgrad> as;
    SmallStep<MODE != kForward> bs;
    UnitEmit<MODE, OT, -1> io;
    float acc[4][8] = {}, db[4] = {};
    pdl_wait();
    as.begin(a, lda, m0, ep.rows, k0);
    bs.begin(b, ldb, n0, ep.cols, k0);
    as.load(k1 - k0);
    bs.load(k1 - k0);
    const int xa = unit_at(warp, 4 * ly), ya = unit_at(warp, 8 * lx), za = unit_at(warp, 8 * lx + 4);   // k = warp + 8 j: 256 j on
    if (warp == 0) io.begin(ep, m0, n0, lane, blockIdx.z * ep.rows);
    int buf = 0;
#pragma unroll 1
    for (int64_t k = k0; k < k1; k += kSmK, buf ^= 1) {
        float* const sa = sm + buf * 2 * kSmK * kSmSide;
        float* const sb = sa + kSmK * kSmSide;
        as.store(sa);
        bs.store(sb);
        __syncthreads();                         // and all are through with the other buffer's step
        if (k + kSmK < k1) {
            as.load(k1 - k - kSmK);
            bs.load(k1 - k - kSmK);
        }
#pragma unroll
        for (int j = 0; j < kSmK / kSmWarps; ++j) {
            const float4 x = ld4(sa + xa + 256 * j), y = ld4(sb + ya + 256 * j), z = ld4(sb + za + 256 * j);
            const float av[4] = {x.x, x.y, x.z, x.w}, bv[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (MODE == kWgrad) db[r] += av[r];
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[r][c] = __fmaf_rn(av[r], bv[c], acc[r][c]);
            }
        }
    }
    __syncthreads();
    float* const unit = sm + warp * kUnitFloats;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        st4(unit + unit_at(4 * ly + r, 8 * lx), make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]));
        st4(unit + unit_at(4 * ly + r, 8 * lx + 4), make_float4(acc[r][4], acc[r][5], acc[r][6], acc[r][7]));
        if (MODE == kWgrad && lx == 0) sums[warp][4 * ly + r] = db[r];
    }
    __syncthreads();
    float4 t = ld4(sm + 4 * threadIdx.x);
#pragma unroll
    for (int w = 1; w < kSmWarps; ++w) {
        const float4 u = ld4(sm + w * kUnitFloats + 4 * threadIdx.x);
        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
    }
    st4(sm + 4 * threadIdx.x, t);
    __syncthreads();
    if (warp == 0) io.run(ep, sm, 1, lane);
    if (MODE == kWgrad && warp == 1 && ep.db && blockIdx.x == 0 && m0 + lane < ep.rows) {
        float s = sums[0][lane];
#pragma unroll
        for (int w = 1; w < kSmWarps; ++w) s += sums[w][lane];
        emit_db<OT>(ep, m0 + lane + blockIdx.z * ep.rows, s);
    }
}

int64_t small_tiles(int64_t rows, int64_t cols) { return ceil_div(rows, kSmSide) * ceil_div(cols, kSmSide); }

template <int MODE, typename OT>
cudaError_t small_as(const SmallProblem& p, const LinEpi& ep, int slabs, int64_t slab_k, cudaStream_t st) {
    const int64_t bx = ceil_div(ep.cols, kSmSide), by = ceil_div(ep.rows, kSmSide);
    if (by > 65535) return cudaErrorInvalidValue;
    return launch(k_small<MODE, OT>, dim3(unsigned(bx), unsigned(by), unsigned(slabs)), dim3(kSmThreads), 0, st, p.a, p.lda, p.b,
                  p.ldb, p.K, slab_k, ep);
}

}  // namespace

// As many slabs as fill the SMs once, of two steps at least.
int small_slabs(int64_t rows, int64_t in, int64_t out) {
    const int64_t by_room = 152 / small_tiles(out, in), by_rows = ceil_div(rows, 2 * kSmK);
    const int64_t s = by_room < by_rows ? by_room : by_rows;
    return s < 1 ? 1 : int(s);
}

// At most two CTAs to an SM, and so many K one after another.  Measured on GB300 (us, this file /
// splitting and tensor cores; forward and dgrad rows x in x out): forward 129 x 64 x 32 2.8 / 8.5,
// 4000 x 64 x 64 4.1 / 9.3, 300^3 7.1 / 11.3, 512^3 13.9 / 10.3, 100 x 1000 x 1000 13.8 / 13.2;
// dgrad 2000 x 64 x 512 9.0 / 11.6, 1000 x 128 x 1000 15.2 / 11.3; wgrad with db 2048 x 64 x 64
// 4.7 / 14.3, 16384 x 64 x 32 6.3 / 19.8, 8000 x 64 x 200 (832 rows a slab) 13.2 / 18.6, 1000 x 300 x 300
// 14.2 / 13.2, 16384 x 128 x 128 25 / 20.
bool use_small(LinMode mode, int64_t rows, int64_t in, int64_t out) {
    const int64_t tiles = mode == kWgrad ? small_tiles(out, in) : small_tiles(rows, mode == kForward ? out : in);
    const int64_t K = mode == kForward ? in : mode == kDgrad ? out : ceil_div(rows, small_slabs(rows, in, out));
    return tiles <= 304 && ceil_div(tiles, 152) * K <= (mode == kWgrad ? 832 : 512);
}

int64_t small_slab_floats(int64_t rows, int64_t in, int64_t out) {
    const int slabs = small_slabs(rows, in, out);
    return use_small(kWgrad, rows, in, out) && slabs > 1 ? int64_t(slabs) * (out * ((in + 7) & ~int64_t(7)) + ((out + 3) & ~int64_t(3))) : 0;
}

cudaError_t launch_small(const SmallProblem& p, cudaStream_t st) {
    if (p.mode == kForward) return small_as<kForward, float>(p, p.epi, 1, p.K, st);
    if (p.mode == kDgrad) return small_as<kDgrad, float>(p, p.epi, 1, p.K, st);
    const int64_t rows = p.epi.rows, cols = p.epi.cols, ld = (cols + 7) & ~int64_t(7);
    const int64_t slab_k = ceil_div(ceil_div(p.K, small_slabs(p.K, cols, rows)), kSmK) * kSmK;
    const int slabs = int(ceil_div(p.K, slab_k));
    if (slabs == 1)
        return p.out_bf16 ? small_as<kWgrad, uint16_t>(p, p.epi, 1, p.K, st) : small_as<kWgrad, float>(p, p.epi, 1, p.K, st);
    LinEpi ep = p.epi;
    float* const db_part = p.partial + slabs * rows * ld;
    ep.out = p.partial;
    ep.ldo = ld;
    ep.db = p.epi.db ? db_part : nullptr;
    ep.accumulate = 0;
    ep.vec = 1;
    const cudaError_t e = small_as<kWgrad, float>(p, ep, slabs, slab_k, st);
    return e != cudaSuccess ? e : launch_join(p.partial, db_part, slabs, rows, cols, ld, p.epi, p.out_bf16, st);
}

}  // namespace fsdp
