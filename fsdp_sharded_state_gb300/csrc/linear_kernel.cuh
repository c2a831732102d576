// linear_kernel.cuh -- the matrix kernel of the linear layers (sm_103a).
//
// D[M, N] = sum over k of A[M, k] B[N, k] on the 5th-generation tensor cores, fp32
// accumulators in TMEM, with the layer's epilogue (bias, activation or its derivative,
// dropout, residual, accumulation) applied before the one rounding to the output type.
//
// Roles of a CTA (12 warps): warp 8 loads the operand tiles with tensor-map copies into a
// ring of stages, warp 9 issues the MMAs, warps 0-7 empty the accumulators, and in wgrad
// warps 10 and 11 add up the columns of the dz tiles for db.  The
// accumulators are double-buffered, so a persistent CTA's epilogue runs beside the next
// tile's products.  Operands keep the row-major layout that the user's tensors have: the
// matrix descriptors take K-major tiles (forward: w and x; dgrad: dz) and MN-major tiles
// (dgrad: w; wgrad: dz and x), so nothing is transposed in memory.
//
// Every wait on an mbarrier is bounded; a role that gives up records it (g_wait_error of
// this translation unit, read by fsdp_check_status), lets copies in flight land and goes
// to the teardown, which every thread of the CTA (and of the cluster) reaches on every path.
#pragma once

#include "internal.hpp"
#include "linear.hpp"
#include "tc5.cuh"

namespace fsdp {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kSumWarps = 2;
constexpr int kLinThreads = (kEpiWarps + 2 + kSumWarps) * 32;
constexpr int kKb = 64;                        // K elements per stage: 128-byte swizzled rows
constexpr int kLinMaxStages = 8;
constexpr int kUnitFloats = 32 * 32;           // an epilogue unit: 32 rows x 32 columns

// ---- 8 consecutive elements, as they lie in memory and as fp32 ------------------------
template <typename T>
struct Raw8 {
    uint4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) r.q[i] = ldu4(reinterpret_cast<const char*>(p) + 16 * i);
    return r;
}
__device__ __forceinline__ void widen(const Raw8<uint16_t>& r, float (&v)[8]) {
    const uint4 u = r.q[0];
    v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
    v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
}
__device__ __forceinline__ void widen(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[4 * i] = __uint_as_float(r.q[i].x); v[4 * i + 1] = __uint_as_float(r.q[i].y);
        v[4 * i + 2] = __uint_as_float(r.q[i].z); v[4 * i + 3] = __uint_as_float(r.q[i].w);
    }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    stu4(p, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    st4(p, make_float4(v[0], v[1], v[2], v[3]));
    st4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16f(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// ---- packed pairs of fp32 --------------------------------------------------------------
// One instruction for two elements: the epilogue is bound by instruction issue.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void unpack(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// The fast base-2 exponential and reciprocal, of both.
__device__ __forceinline__ F2 exp2_fast(F2 x) {
    float a, b;
    unpack(x, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2(a, b);
}
__device__ __forceinline__ F2 rcp_fast(F2 x) {
    float a, b;
    unpack(x, a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return f2(a, b);
}

// ---- activations (fp32) --------------------------------------------------------------
// gelu(z) = z Phi(z), gelu'(z) = Phi(z) + z exp(-z^2/2) / sqrt(2 pi);
// silu(z) = z s, silu'(z) = s (1 + z (1 - s)), s = 1 / (1 + exp(-z)).
// For fp32 results, CUDA's erff and expf.  For bf16 results (rounded to 2^-8 afterwards)
// the fast exponential and reciprocal, in pairs, and for Phi formula 7.1.26 of Abramowitz
// and Stegun, Handbook of Mathematical Functions: erf(x) = 1 - (a1 t + .. + a5 t^5) exp(-x^2),
// t = 1 / (1 + 0.3275911 x), for x >= 0, error at most 1.5e-7; its exponential is also the
// derivative's.  A tile of 256 x 256 leaves the epilogue 16,000 clocks beside the products of
// K = 2048: 64 issue slots per element.  With CUDA's erff, expf and division unrolled over a
// unit, its code did not fit the instruction caches, and the tile's epilogue took 26,000
// clocks even with no activation asked for.
struct PhiExp {
    F2 phi, e;                 // Phi(z), exp(-z^2 / 2)
};
__device__ __forceinline__ PhiExp phi_exp(float z0, float z1) {
    const F2 x = f2(fabsf(z0), fabsf(z1)) * f2(0.70710678118654752f);
    PhiExp r;
    r.e = exp2_fast(x * x * f2(-1.4426950408889634f));
    const F2 t = rcp_fast(fma(f2(0.3275911f), x, f2(1.f)));
    F2 q = fma(t, f2(0.5f * 1.061405429f), f2(0.5f * -1.453152027f));
    q = fma(t, q, f2(0.5f * 1.421413741f));
    q = fma(t, q, f2(0.5f * -0.284496736f));
    q = fma(t, q, f2(0.5f * 0.254829592f));
    // (1 - erf(x)) / 2 = t q e, so Phi = 1/2 +- (1/2 - t q e)
    float a, b;
    unpack(fma(t * q * f2(-1.f), r.e, f2(0.5f)), a, b);
    r.phi = f2(copysignf(a, z0), copysignf(b, z1)) + f2(0.5f);
    return r;
}
__device__ __forceinline__ F2 sigmoid(F2 z) { return rcp_fast(exp2_fast(z * f2(-1.4426950408889634f)) + f2(1.f)); }

template <bool FAST, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    if (act == FSDP_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];              // NaN stays NaN
    } else if (act == FSDP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += FAST ? 2 : 1) {
            if constexpr (FAST) unpack(f2(v[i], v[i + 1]) * phi_exp(v[i], v[i + 1]).phi, v[i], v[i + 1]);
            else v[i] *= __fmaf_rn(0.5f, erff(v[i] * 0.70710678118654752f), 0.5f);
        }
    } else if (act == FSDP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; i += FAST ? 2 : 1) {
            if constexpr (FAST) {
                const F2 z = f2(v[i], v[i + 1]);
                unpack(z * sigmoid(z), v[i], v[i + 1]);
            } else {
                v[i] = v[i] / (1.f + expf(-v[i]));
            }
        }
    }
}
// v *= act'(z)
template <bool FAST, int N>
__device__ __forceinline__ void activate_grad(float (&v)[N], const float (&z)[N], int act) {
    if (act == FSDP_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = z[i] > 0.f ? v[i] : 0.f;
    } else if (act == FSDP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i += FAST ? 2 : 1) {
            if constexpr (FAST) {
                const PhiExp p = phi_exp(z[i], z[i + 1]);
                unpack(f2(v[i], v[i + 1]) * fma(f2(z[i], z[i + 1]) * f2(0.39894228040143268f), p.e, p.phi), v[i], v[i + 1]);
            } else {
                const float phi = __fmaf_rn(0.5f, erff(z[i] * 0.70710678118654752f), 0.5f);
                v[i] *= __fmaf_rn(z[i] * 0.39894228040143268f, expf(-0.5f * z[i] * z[i]), phi);
            }
        }
    } else if (act == FSDP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; i += FAST ? 2 : 1) {
            if constexpr (FAST) {
                const F2 x = f2(z[i], z[i + 1]), s = sigmoid(x);
                unpack(f2(v[i], v[i + 1]) * (s * fma(x, fma(s, f2(-1.f), f2(1.f)), f2(1.f))), v[i], v[i + 1]);
            } else {
                const float s = 1.f / (1.f + expf(-z[i]));
                v[i] *= s * __fmaf_rn(z[i], 1.f - s, 1.f);
            }
        }
    }
}

template <typename OT>
__device__ __forceinline__ void emit_db(const LinEpi& ep, int64_t c, float t) {
    OT* const p = static_cast<OT*>(ep.db) + c;
    store1(p, ep.accumulate ? t + load1(p) : t);
}

// A unit in shared memory: [32 rows][32 columns] fp32, the 16-byte groups of row r at
// group index g ^ (r & 7), so that both ways of writing it (a lane holds a row, a lane
// holds a column) and the row-wise reads are free of bank conflicts.
__device__ __forceinline__ int unit_at(int r, int c) { return r * 32 + ((((c >> 2) ^ (r & 7)) << 2) | (c & 3)); }

// The epilogue of one unit from shared memory: 4 lanes per row, 8 columns per lane, 8 rows at a
// time; what it reads of memory (the addend: the residual, or what wgrad accumulates to; the
// pre-activation) one step of 8 rows ahead, the first step by begin(), which a caller runs
// before it fetches the accumulators.  EP: the activation (+ 4 with dropout) that the kernel is
// compiled for, or -1 for the call's.  Jumping over what a call does not use costs more than
// computing it: the loop outgrows the innermost instruction cache, and a unit with neither took
// 2,150 clocks with EP = -1 where 1,150 do.
template <int MODE, typename OT, int EP>
struct UnitEmit {
    static constexpr bool FAST = sizeof(OT) == 2;
    static __device__ __forceinline__ int act(const LinEpi& ep) { return EP >= 0 ? EP & 3 : ep.act; }
    static __device__ __forceinline__ bool drop(const LinEpi& ep) { return EP >= 0 ? EP >= 4 : ep.drop.on != 0; }
    OT* out;
    const OT* add;
    OT* z;
    int64_t add_step, z_step, row0, col0, shift;
    int n_it;                                    // steps of 8 rows; -1: not by vectors
    Raw8<OT> aq, zq;

    // shift: rows that out starts further down (a slab of partial sums)
    __device__ __forceinline__ void begin(const LinEpi& ep, int64_t row0_, int64_t col0_, int lane, int64_t shift_ = 0) {
        row0 = row0_;
        col0 = col0_;
        shift = shift_;
        n_it = -1;
        if (!ep.vec || ep.cols - col0 < 32) return;
        const int64_t col = col0 + (lane & 3) * 8, row1 = row0 + (lane >> 2);
        n_it = ep.rows > row1 ? (ep.rows - row1 >= 32 ? 4 : int((ep.rows - row1 + 7) >> 3)) : 0;
        out = static_cast<OT*>(ep.out) + (row1 + shift) * ep.ldo + col;
        add = MODE == kWgrad ? (ep.accumulate ? out : nullptr)
              : ep.residual  ? static_cast<const OT*>(ep.residual) + row1 * ep.ldr + col
                             : nullptr;
        add_step = 8 * (MODE == kWgrad ? ep.ldo : ep.ldr);
        z = MODE != kWgrad && ep.preact ? static_cast<OT*>(ep.preact) + row1 * ep.ldz + col : nullptr;
        z_step = 8 * ep.ldz;
        if (add && n_it > 0) aq = load_raw(add);
        if (MODE == kDgrad && z && n_it > 0) zq = load_raw(z);
    }

    // Adds the `slots` copies of the unit (kUnitFloats apart, in order) and emits it.
    __device__ __forceinline__ void run(const LinEpi& ep, const float* unit, int slots, int lane) {
        if (n_it < 0) {
            by_columns(ep, unit, slots, lane);
            return;
        }
        const int64_t col = col0 + (lane & 3) * 8;
        DropCol dc[2] = {};                      // the generator's column products, for all rows of the unit
        uint32_t row_hi = 0, row_u = 0;
        float bias[8] = {};
        if (MODE == kForward && ep.bias && n_it > 0) widen(load_raw(static_cast<const OT*>(ep.bias) + col), bias);
#pragma unroll 1
        for (int it = 0; it < n_it; ++it) {
            const int r = it * 8 + (lane >> 2);
            const float* p = unit + unit_at(r, (lane & 3) * 8);
            const float* q = unit + unit_at(r, (lane & 3) * 8 + 4);
            float4 a = ld4(p), b = ld4(q);
#pragma unroll 1
            for (int s = 1; s < slots; ++s) {
                const float4 c = ld4(p + s * kUnitFloats), d = ld4(q + s * kUnitFloats);
                a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
                b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
            }
            float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const Raw8<OT> add_c = aq, z_c = zq;
            if (it + 1 < n_it) {
                if (add) aq = load_raw(add + (it + 1) * add_step);
                if (MODE == kDgrad && z) zq = load_raw(z + (it + 1) * z_step);
            }
            if constexpr (MODE == kForward) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += bias[i];
                if (z) store8(z + it * z_step, v);
                activate<FAST, 8>(v, act(ep));
            }
            if constexpr (MODE != kWgrad) {
                if (drop(ep)) {
                    const uint64_t gr = uint64_t(row0 + r + ep.drop.row0);
                    if (it == 0 || uint32_t(gr >> 32) != row_hi) {
                        row_hi = uint32_t(gr >> 32);
                        dc[0] = drop_col(ep.drop, uint32_t(col >> 2), row_hi);
                        dc[1] = drop_col(ep.drop, uint32_t(col >> 2) + 1, row_hi);
                        row_u = __umulhi(0xCD9E8D57u, row_hi);
                    }
                    const DropRow dr = drop_row(ep.drop, uint32_t(gr), row_u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 w = drop_words(ep.drop, dr, dc[h]);
                        v[4 * h] = drop1(ep.drop, w.x, v[4 * h]);
                        v[4 * h + 1] = drop1(ep.drop, w.y, v[4 * h + 1]);
                        v[4 * h + 2] = drop1(ep.drop, w.z, v[4 * h + 2]);
                        v[4 * h + 3] = drop1(ep.drop, w.w, v[4 * h + 3]);
                    }
                }
            }
            float t[8];
            if constexpr (MODE == kDgrad) {
                if (z) {
                    widen(z_c, t);
                    activate_grad<FAST, 8>(v, t, act(ep));
                }
            }
            if (add) {
                widen(add_c, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += t[i];
            }
            store8(out, v);
            out += 8 * ep.ldo;
        }
    }

    // Any alignment, and a ragged right edge: a lane per column, 8 rows at a time.
    __device__ __forceinline__ void by_columns(const LinEpi& ep, const float* unit, int slots, int lane) const {
        const int64_t c = col0 + lane;
        const bool in = c < ep.cols;
        const float bias = MODE == kForward && ep.bias && in ? load1(static_cast<const OT*>(ep.bias) + c) : 0.f;
        OT* o = static_cast<OT*>(ep.out) + (row0 + shift) * ep.ldo + c;
        const OT* addp = MODE == kWgrad ? (ep.accumulate ? o : nullptr)
                        : ep.residual  ? static_cast<const OT*>(ep.residual) + row0 * ep.ldr + c
                                       : nullptr;
        const int64_t add_ld = MODE == kWgrad ? ep.ldo : ep.ldr;
        OT* zp = MODE != kWgrad && ep.preact ? static_cast<OT*>(ep.preact) + row0 * ep.ldz + c : nullptr;
#pragma unroll 1
        for (int r0 = 0; r0 < 32 && row0 + r0 < ep.rows; r0 += 8) {
            const int n = !in ? 0 : ep.rows - row0 - r0 >= 8 ? 8 : int(ep.rows - row0 - r0);
            float v[8], a[8], zs[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] = addp && i < n ? load1(addp + (r0 + i) * add_ld) : 0.f;
                zs[i] = MODE == kDgrad && zp && i < n ? load1(zp + (r0 + i) * ep.ldz) : 0.f;
                v[i] = unit[unit_at(r0 + i, lane)];
            }
#pragma unroll 1
            for (int s = 1; s < slots; ++s) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += unit[unit_at(r0 + i, lane) + s * kUnitFloats];
            }
            if constexpr (MODE == kForward) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] += bias;
                    if (zp && i < n) store1(zp + (r0 + i) * ep.ldz, v[i]);
                }
                activate<FAST, 8>(v, act(ep));
            }
            if constexpr (MODE != kWgrad) {
                if (drop(ep)) {
                    // lane l draws the blocks of columns 4 (l mod 8) on of rows l / 8 and l / 8 + 4, as keep
                    // bits; column `lane` of row i is bit lane mod 4 of what lane 8 (i mod 4) + lane / 4 drew
                    uint32_t keep = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 w = drop_words(ep.drop, row0 + r0 + (lane >> 3) + 4 * h, (col0 >> 2) + (lane & 7));
                        keep |= (uint32_t(w.x >= ep.drop.thr) | uint32_t(w.y >= ep.drop.thr) << 1 |
                                 uint32_t(w.z >= ep.drop.thr) << 2 | uint32_t(w.w >= ep.drop.thr) << 3) << (4 * h);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b = __shfl_sync(0xffffffffu, keep, 8 * i + (lane >> 2)) >> (lane & 3);
                        v[i] = b & 1 ? v[i] * ep.drop.scale : 0.f;
                        v[i + 4] = b >> 4 & 1 ? v[i + 4] * ep.drop.scale : 0.f;
                    }
                }
            }
            if constexpr (MODE == kDgrad) {
                if (zp) activate_grad<FAST, 8>(v, zs, act(ep));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) store1(o + (r0 + i) * ep.ldo, v[i] + a[i]);
        }
    }
};

// 16 bf16 elements in one access of 32 bytes (32-byte aligned).
struct Raw16 {
    uint32_t w[8];
};
__device__ __forceinline__ Raw16 load_raw16(const uint16_t* p) {
    Raw16 r;
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ void widen(const Raw16& r, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = bf16lo(r.w[i]);
        v[2 * i + 1] = bf16hi(r.w[i]);
    }
}
__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 16 bf16 elements that start o elements into a 16-byte window (0 <= o < 8), as the three
// windows that hold them, the third only where it is needed.
struct Win16 {
    uint32_t w[12];
};
__device__ __forceinline__ int window_offset(const uint16_t* p) { return int(reinterpret_cast<uintptr_t>(p) & 15) >> 1; }
__device__ __forceinline__ Win16 load_win16(const uint16_t* p) {
    const uint16_t* const a = p - window_offset(p);
    Win16 r;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (k < 2 || a != p) q = ldu4(a + 8 * k);
        r.w[4 * k] = q.x; r.w[4 * k + 1] = q.y; r.w[4 * k + 2] = q.z; r.w[4 * k + 3] = q.w;
    }
    return r;
}
__device__ __forceinline__ void widen(const Win16& r, int o, float (&v)[16]) {
    uint32_t u[11];                              // by half a word, then by 2 words, then by 1
#pragma unroll
    for (int i = 0; i < 11; ++i) u[i] = __funnelshift_r(r.w[i], r.w[i + 1], 16 * (o & 1));
#pragma unroll
    for (int i = 0; i < 9; ++i) u[i] = o & 4 ? u[i + 2] : u[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = o & 2 ? u[i + 1] : u[i];
        v[2 * i] = bf16lo(w);
        v[2 * i + 1] = bf16hi(w);
    }
}
// The other way: groups of 16 elements that follow one another in memory from p on, written as
// whole 16-byte windows; the elements before the first and after the last whole window, which
// neighbours share, in pieces of 8, 4 and 2 bytes.
struct WinOut {
    uint16_t* at;              // the window that the next group starts in
    int o;                     // elements of it that are already there
    uint32_t carry[4];         // those, where an earlier group left them
    bool first;

    __device__ __forceinline__ void begin(uint16_t* p) {
        o = window_offset(p);
        at = p - o;
        carry[0] = carry[1] = carry[2] = carry[3] = 0;
        first = true;
    }
    // elements [lo, 8) or [0, hi) of a window, from its words
    __device__ __forceinline__ static void tail(uint16_t* a, const uint32_t (&w)[4], int lo) {
        if (lo & 1) a[lo] = uint16_t((lo & 2 ? (lo & 4 ? w[3] : w[1]) : (lo & 4 ? w[2] : w[0])) >> 16);
        const int e = (lo + 1) & ~1;             // even
        if (e & 2) *reinterpret_cast<uint32_t*>(a + e) = e & 4 ? w[3] : w[1];
        const int f = (e + 3) & ~3;              // 0, 4 or 8; 0 only where the window is whole
        if (f == 4) *reinterpret_cast<uint2*>(a + 4) = make_uint2(w[2], w[3]);
    }
    __device__ __forceinline__ static void head(uint16_t* a, const uint32_t (&w)[4], int hi) {
        if (hi & 4) *reinterpret_cast<uint2*>(a) = make_uint2(w[0], w[1]);
        if (hi & 2) *reinterpret_cast<uint32_t*>(a + (hi & 4)) = hi & 4 ? w[2] : w[0];
        if (hi & 1) a[hi & 6] = uint16_t(hi & 4 ? (hi & 2 ? w[3] : w[2]) : (hi & 2 ? w[1] : w[0]));
    }
    __device__ __forceinline__ void put(const float (&v)[16]) {
        uint32_t t[12];                          // the elements shifted o up: by half a word, 1 word, 2 words
        uint32_t prev = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            t[i] = o & 1 ? __funnelshift_l(prev, x, 16) : x;
            prev = x;
        }
        t[8] = o & 1 ? prev >> 16 : 0;
        t[9] = t[10] = t[11] = 0;
#pragma unroll
        for (int i = 11; i >= 0; --i) {
            if (i <= 9) t[i] = o & 2 ? (i >= 1 ? t[i - 1] : 0) : t[i];
        }
#pragma unroll
        for (int i = 11; i >= 0; --i) t[i] = o & 4 ? (i >= 2 ? t[i - 2] : 0) : t[i];
        const uint32_t w0[4] = {t[0] | carry[0], t[1] | carry[1], t[2] | carry[2], t[3] | carry[3]};
        if (first && o) tail(at, w0, o);
        else stu4(at, make_uint4(w0[0], w0[1], w0[2], w0[3]));
        stu4(at + 8, make_uint4(t[4], t[5], t[6], t[7]));
        carry[0] = t[8]; carry[1] = t[9]; carry[2] = t[10]; carry[3] = t[11];
        at += 16;
        first = false;
    }
    __device__ __forceinline__ void end() {
        if (!first && o) head(at, carry, o);
    }
};

// The epilogue straight from the accumulators, a lane per row: no trip through shared memory,
// whose bandwidth the products of a CTA pair use up.  For bf16 results of persistent tiles.  An
// access of a warp touches 32 lines whatever its width, so rows aligned to 32 bytes (ALIGNED)
// are read and written by whole 32-byte sectors; rows that start anywhere by whole 16-byte
// windows, the elements shifted into place in registers (through shared memory and by single
// elements, a lane per column, the tile took 30,000 clocks).  The warp takes units of 32
// columns, STEP apart from col0 on, while they lie wholly inside the matrix, NU at most, and
// returns how many; a unit's two halves are read (residual, pre-activation) while the unit before it is
// computed.  dcol: the generator's column products of the units' columns, in shared memory;
// dr: the lane's row's.
template <int MODE, int EP, int NU, bool ALIGNED>
struct RowsEmit {
    using In = typename std::conditional<ALIGNED, Raw16, Win16>::type;
    static constexpr int STEP = ALIGNED ? 64 : 32;
    uint16_t* out;
    const uint16_t* add;
    uint16_t* z;
    const uint16_t* bias;
    int units;
    bool in;
    In aq[2], zq[2];

    __device__ __forceinline__ static In load(const uint16_t* p) {
        if constexpr (ALIGNED) return load_raw16(p);
        else return load_win16(p);
    }
    __device__ __forceinline__ static void value(const In& r, const uint16_t* p, float (&v)[16]) {
        if constexpr (ALIGNED) widen(r, v);
        else widen(r, window_offset(p), v);      // the same for all groups of a row: 16 elements are two windows
    }

    // Before the accumulators are there: the first unit's reads.
    __device__ __forceinline__ void begin(const LinEpi& ep, int64_t row, int64_t col0) {
        in = row < ep.rows;
        const int64_t left = ep.cols - col0;
        units = left < 32 ? 0 : (left - 32) / STEP + 1 < NU ? int((left - 32) / STEP + 1) : NU;
        out = static_cast<uint16_t*>(ep.out) + row * ep.ldo + col0;
        add = MODE == kWgrad ? (ep.accumulate ? out : nullptr)
              : ep.residual  ? static_cast<const uint16_t*>(ep.residual) + row * ep.ldr + col0
                             : nullptr;
        z = MODE != kWgrad && ep.preact ? static_cast<uint16_t*>(ep.preact) + row * ep.ldz + col0 : nullptr;
        bias = MODE == kForward && ep.bias ? static_cast<const uint16_t*>(ep.bias) + col0 : nullptr;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            aq[g] = zq[g] = In{};
            if (add && in && units > 0) aq[g] = load(add + 16 * g);
            if (MODE == kDgrad && z && in && units > 0) zq[g] = load(z + 16 * g);
        }
    }

    __device__ __forceinline__ int run(const LinEpi& ep, uint32_t acc, const DropRow& dr, const DropCol* dcol) {
        const int act = EP >= 0 ? EP & 3 : ep.act;
        const bool drop = MODE != kWgrad && (EP >= 0 ? EP >= 4 : ep.drop.on != 0);
        WinOut wo, wz;
        if constexpr (!ALIGNED) {
            wo.begin(out);
            if (MODE == kForward && z) wz.begin(z);
        }
        Acc16 next;                                              // the accumulators of the half to come
        if (units > 0) tmem_ld16_async(acc, next);
#pragma unroll 1
        for (int u = 0; u < units; ++u) {
            const bool more = in && u + 1 < units;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int c = STEP * u + 16 * g;
                float v[16], t[16];
                tmem_wait_ld16(next, v);
                if (g == 0 || u + 1 < units) tmem_ld16_async(acc + c + (g == 0 ? 16 : STEP - 16), next);
                if constexpr (MODE == kForward) {
                    if (bias) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float b[8];
                            if constexpr (ALIGNED) {
                                widen(load_raw(bias + c + 8 * h), b);
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i) b[i] = load1(bias + c + 8 * h + i);
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[8 * h + i] += b[i];
                        }
                    }
                    if (z && in) {
                        if constexpr (ALIGNED) store16(z + c, v);
                        else wz.put(v);
                    }
                    activate<true, 16>(v, act);
                }
                if (drop) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint4 q = ldu4(dcol + 8 * u + 4 * g + b);
                        const uint4 w = drop_words(ep.drop, dr, DropCol{q.x, q.y, q.z, q.w});
                        v[4 * b] = drop1(ep.drop, w.x, v[4 * b]);
                        v[4 * b + 1] = drop1(ep.drop, w.y, v[4 * b + 1]);
                        v[4 * b + 2] = drop1(ep.drop, w.z, v[4 * b + 2]);
                        v[4 * b + 3] = drop1(ep.drop, w.w, v[4 * b + 3]);
                    }
                }
                if constexpr (MODE == kDgrad) {
                    if (z) {
                        value(zq[g], z, t);
                        if (more) zq[g] = load(z + c + STEP);
                        activate_grad<true, 16>(v, t, act);
                    }
                }
                if (add) {
                    value(aq[g], add, t);
                    if (more) aq[g] = load(add + c + STEP);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += t[i];
                }
                if (in) {
                    if constexpr (ALIGNED) store16(out + c, v);
                    else wo.put(v);
                }
            }
        }
        if constexpr (!ALIGNED) {
            if (in) {
                wo.end();
                if (MODE == kForward && z) wz.end();
            }
        }
        return units;
    }
};

// wgrad's fp32 epilogue from the sums in registers, a lane per row, 32-byte aligned rows: the
// columns col0 + 64 u on are written, or added to what is there, which is read further and
// further ahead into the registers that the written sums leave (the staged path, one step of 8
// rows ahead, waits out 16 latencies of memory per tile).
struct Raw8f {
    float v[8];
};
__device__ __forceinline__ void load_8f(const float* p, Raw8f& r) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(r.v[0]), "=f"(r.v[1]), "=f"(r.v[2]), "=f"(r.v[3]), "=f"(r.v[4]), "=f"(r.v[5]), "=f"(r.v[6]), "=f"(r.v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store_8f(float* p, const Raw8f& r) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(r.v[0]), "f"(r.v[1]), "f"(r.v[2]), "f"(r.v[3]),
                 "f"(r.v[4]), "f"(r.v[5]), "f"(r.v[6]), "f"(r.v[7])
                 : "memory");
}
template <int NU>
__device__ __forceinline__ void emit_sums(const LinEpi& ep, const float (&sum)[NU][32], int64_t row, int64_t col0) {
    if (row >= ep.rows) return;
    float* const out = static_cast<float*>(ep.out) + row * ep.ldo + col0;
    constexpr int G = 4 * NU, FIRST = 2;         // groups of 8 columns; read ahead at the start, one more per group written
    Raw8f old[G];
    if (ep.accumulate) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int k = g == 0 ? 0 : 2 * g + FIRST - 2; k < 2 * g + FIRST; ++k)
                if (k < G) load_8f(out + 64 * (k / 4) + 8 * (k % 4), old[k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) old[g].v[e] += sum[g / 4][8 * (g % 4) + e];
            store_8f(out + 64 * (g / 4) + 8 * (g % 4), old[g]);
        }
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            Raw8f r;
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = sum[g / 4][8 * (g % 4) + e];
            store_8f(out + 64 * (g / 4) + 8 * (g % 4), r);
        }
    }
}

// ---- column sums of dz (wgrad's db) ---------------------------------------------------
// Where K is split: two warps add up the dz tiles that the products of the first column of tiles
// read anyway, from shared memory.  A tile (one plane) is two chunks of 64
// columns, each 64 rows of 128 bytes whose 16-byte groups are swizzled: group p of row r holds
// columns 8 (p ^ (r mod 8)) on.  A warp takes a chunk; lane l reads group l mod 8 of rows l / 8
// + 4 h + 8 j: the same columns for all j.  A tile's 8 rows are added in a tree before they
// meet the running sums.
struct ColSum {
    float v[2][8];
};
template <int PL>
__device__ __forceinline__ void colsum_row(float (&x)[8], const unsigned char* p, int plane_bytes) {
    widen(load_raw(reinterpret_cast<const uint16_t*>(p)), x);
    if constexpr (PL == 3) {                                 // hi + (mid + lo): both sums exact
        float a[8], b[8];
        widen(load_raw(reinterpret_cast<const uint16_t*>(p + plane_bytes)), a);
        widen(load_raw(reinterpret_cast<const uint16_t*>(p + 2 * plane_bytes)), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += a[e] + b[e];
    }
}
template <int PL>
__device__ __forceinline__ void colsum_add(ColSum& s, const unsigned char* chunk, int plane_bytes, int lane) {
    const unsigned char* p = chunk + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float t[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j) colsum_row<PL>(x[j], p + h * 512 + (4 * k + j) * 1024, plane_bytes);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[k][e] = (x[0][e] + x[1][e]) + (x[2][e] + x[3][e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[h][e] += t[0][e] + t[1][e];
    }
}
// Column u * 8 + e of the chunk to t[e] of lane u < 8, in a fixed order.
__device__ __forceinline__ void colsum_lanes(const ColSum& s, float (&t)[8], int lane) {
    const int row = lane >> 3, u = lane & 7;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        t[e] = __shfl_sync(0xffffffffu, s.v[0][e], (row << 3) | (u ^ row)) +
               __shfl_sync(0xffffffffu, s.v[1][e], (row << 3) | (u ^ (row + 4)));
        t[e] += __shfl_xor_sync(0xffffffffu, t[e], 8);
        t[e] += __shfl_xor_sync(0xffffffffu, t[e], 16);
    }
}

// For the CTA pairs: 64 columns (from col) of 64 rows of dz (from row, `rows` in all) added to
// the lane's sums straight from memory, which the tiles' own copies have just brought into L2.
// (From the shared-memory stages it held each of them back from its next load by more than
// the ring of stages covers: dz^T x of 16384 x 2048 x 2048 took 111 us against 78 without db.)
// Lane l holds columns E (l mod L) on, L = 64 / E lanes to a row.
template <typename T>
struct RowSum {
    static constexpr int E = 16 / sizeof(T), L = 64 / E;
    float v[E];

    __device__ __forceinline__ static void wide(const uint4& q, float (&x)[E]) {
        if constexpr (E == 8) {
            Raw8<uint16_t> r;
            r.q[0] = q;
            widen(r, x);
        } else {
            x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y);
            x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
        }
    }
    __device__ __forceinline__ void add(const T* dz, int64_t ld, int64_t row, int64_t rows, int64_t col, int64_t cols, bool vec, int lane) {
        constexpr int R = 32 / L, N = 64 / R, B = 16;            // rows of a load; loads; of a batch
        const int64_t c = col + (lane % L) * E;
#pragma unroll 1
        for (int b = 0; b < N; b += B) {
            const int64_t r0 = row + b * R + lane / L;
            if (vec && col + 64 <= cols && row + 64 <= rows) {
                uint4 q[B];
#pragma unroll
                for (int i = 0; i < B; ++i) q[i] = ldu4(dz + (r0 + i * R) * ld + c);
#pragma unroll
                for (int i = 0; i < B; i += 4) {
                    float x[4][E];
#pragma unroll
                    for (int k = 0; k < 4; ++k) wide(q[i + k], x[k]);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] += (x[0][e] + x[1][e]) + (x[2][e] + x[3][e]);
                }
            } else {                                         // any alignment, ragged ends
#pragma unroll 1
                for (int i = 0; i < B; ++i) {
                    const int64_t r = r0 + i * R;
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] += r < rows && c + e < cols ? load1(dz + r * ld + c + e) : 0.f;
                }
            }
        }
    }
    // Lane l < L: the sums of its columns over the warp.
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int m = L; m < 32; m <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], m);
        }
    }
};

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
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BROWS * 128;
    static constexpr int STAGE = PL * (A_BYTES + B_BYTES);
    // the epilogue's shared memory: a unit per warp, or the join's slots
    static constexpr int EPI = SPLIT ? (BN >= 128 ? 64 : 32) * 1024 : kEpiWarps * kUnitFloats * 4;
    static constexpr int MORE = SPLIT && MODE == kWgrad ? 2560 : 2048;   // alignment, barriers, a split's column sums
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
struct LinShape {
    int32_t m_tiles, n_tiles, n_kb, splits, slabs;
};

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
    const uint32_t summed = tmem_word + 8;       // wgrad: a stage's dz tile has been added
    static_assert(8 * (3 * kLinMaxStages + 6) <= 256, "barriers");
    float* const db_part = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE + C::EPI + 256);   // SPLIT: [128]
    const bool leader = C::CG == 1 || rank == 0;

    if (warp == 0) tmem_alloc<C::CG>(tmem_word, C::TMEM);
    if (tid == kEpiWarps * 32) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
            mbar_init(summed + 8 * s, kSumWarps);
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

    // Tiles in bands of 8 along M, N outer inside a band: concurrently running tiles share
    // operand rows in L2.
    auto tile_at = [&](int t, int& mt, int& nt) {
        const int band = 8 * sh.n_tiles, g = t / band, first = g * 8;
        const int high = sh.m_tiles - first < 8 ? sh.m_tiles - first : 8;
        const int r = t - g * band;
        mt = first + r % high;
        nt = r / high;
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
            uint32_t adding = 0, parity = 0;             // per stage: its tile is being added; phase of `summed`
            for (int t = cluster; ok && t < n_tiles; t += n_clusters) {
                int mt, nt;
                tile_at(t, mt, nt);
                const int m0 = (mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128;
                const int n0 = nt * C::BN + (C::CG == 2 ? int(rank) * C::BROWS : 0);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % C::STAGES, use = it / C::STAGES;
                    if (use > 0 && !mbar_wait_bounded(empty + 8 * s, (use - 1) & 1, wait_ns)) {
                        ok = false;
                        break;
                    }
                    if (C::SPLIT && C::MODE == kWgrad && (adding >> s & 1)) {
                        if (!mbar_wait_bounded(summed + 8 * s, parity >> s & 1, wait_ns)) {
                            ok = false;
                            break;
                        }
                        parity ^= 1u << s;
                        adding ^= 1u << s;
                    }
                    if (C::SPLIT && C::MODE == kWgrad && ep.db && nt == 0) adding |= 1u << s;
                    if (elect_one()) {
                        if (leader) mbar_arrive_tx(full + 8 * s, C::CG * C::STAGE);
                        const uint32_t bar = C::CG == 2 ? map_rank(full + 8 * s, 0) : full + 8 * s;
                        const uint32_t st = smem_addr(smem + s * C::STAGE);
#pragma unroll
                        for (int p = 0; p < C::PL; ++p) {
                            const uint32_t a = st + p * C::A_BYTES, b = st + C::PL * C::A_BYTES + p * C::B_BYTES;
                            if constexpr (C::A_MN) {
                                tma_load<C::CG>(a, &map_a, m0, kb * kKb, p, bar);
                                tma_load<C::CG>(a + 8192, &map_a, m0 + 64, kb * kKb, p, bar);
                            } else {
                                tma_load<C::CG>(a, &map_a, kb * kKb, m0, p, bar);
                            }
                            if constexpr (C::B_MN) {
#pragma unroll
                                for (int c = 0; c < C::BROWS / 64; ++c)
                                    tma_load<C::CG>(b + c * 8192, &map_b, n0 + c * 64, kb * kKb, p, bar);
                            } else {
                                tma_load<C::CG>(b, &map_b, kb * kKb, n0, p, bar);
                            }
                        }
                    }
                    __syncwarp();
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
                constexpr uint32_t idesc = mma_idesc(128 * C::CG, C::BN, C::A_MN, C::B_MN);
                // 16 K elements on: 32 bytes along a K-major row, 16 rows of an MN-major tile
                constexpr uint32_t a_step = C::A_MN ? 2048 / 16 : 32 / 16, b_step = C::B_MN ? 2048 / 16 : 32 / 16;
                const uint64_t da0 = smem_desc(smem_addr(smem), C::A_MN ? 8192 : 16, 1024);
                const uint64_t db0 = smem_desc(smem_addr(smem) + C::PL * C::A_BYTES, C::B_MN ? 8192 : 16, 1024);
                bool ok = true;
                uint32_t it = 0, ac = 0;
                for (int t = cluster; ok && t < n_tiles; t += n_clusters) {
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
            const int chunk_at = warp - (kEpiWarps + 2);
            if (C::MODE == kWgrad && C::SPLIT && ep.db) {
                // a stage is read once it is loaded, and loaded again once it has been added
                int mt, nt;
                tile_at(cluster, mt, nt);
                bool ok = true;
                ColSum db = {};
                for (int kb = kb0; nt == 0 && kb < kb1; ++kb) {
                    const uint32_t it = uint32_t(kb - kb0), s = it % C::STAGES;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(full + 8 * s, (it / C::STAGES) & 1, wait_ns));
                    if (!ok) break;
                    colsum_add<C::PL>(db, smem + s * C::STAGE + chunk_at * 8192, C::A_BYTES, lane);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(summed + 8 * s);
                }
                float v[8];
                colsum_lanes(db, v, lane);
                if (lane < 8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) db_part[chunk_at * 64 + lane * 8 + e] = v[e];
                }
                if (!ok && lane == 0) atomicOr(&g_wait_error, 1u);
            }
            if constexpr (C::MODE == kWgrad && !C::SPLIT) {
                // the tiles of a row of tiles belong to the same columns of dz: the first db_parts of
                // them share out the K steps, every db_parts-th each
                using DT = typename std::conditional<C::PL == 3, float, uint16_t>::type;
                using RS = RowSum<DT>;
                for (int t = cluster; ep.db && t < n_tiles; t += n_clusters) {
                    int mt, nt;
                    tile_at(t, mt, nt);
                    if (nt >= ep.db_parts) continue;
                    const int64_t col = int64_t(mt * C::CG + int(rank)) * 128 + chunk_at * 64;
                    RS db = {};
                    for (int kb = nt; kb < sh.n_kb && col < ep.rows; kb += ep.db_parts)
                        db.add(static_cast<const DT*>(ep.dz), ep.lddz, int64_t(kb) * kKb, ep.dz_rows, col, ep.rows, ep.dz_vec, lane);
                    db.join();
                    if (lane < RS::L) {
#pragma unroll
                        for (int e = 0; e < RS::E; ++e) {
                            const int64_t c = col + lane * RS::E + e;
                            if (c >= ep.rows) break;
                            if (ep.db_parts > 1) ep.db_sums[nt * ep.rows + c] = db.v[e];
                            else emit_db<typename C::OT>(ep, c, db.v[e]);
                        }
                    }
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
        auto group = [&](int jj) { return C::DIRECT && C::ANY ? half * NJ + jj : 2 * jj + half; };
        bool ok = true;
        uint32_t ac = 0;
        for (int t = cluster; ok && t < n_tiles; t += n_clusters) {
            int mt, nt;
            tile_at(t, mt, nt);
            const int64_t m0 = int64_t(mt * C::CG + (C::CG == 2 ? int(rank) : 0)) * 128 + q * 32;
            const int64_t n0 = int64_t(nt) * C::BN;
            float sum[C::CH ? NJ : 1][32];
            if constexpr (C::CH != 0) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[j][i] = 0.f;
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
                RowsEmit<C::MODE, C::EP, NJ, !C::ANY> rows;
                bool direct = C::DIRECT;
                if constexpr (C::DIRECT) rows.begin(ep, m0 + lane, n0 + group(0) * 32);
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
                    if (group(jj) * 32 < C::BN) {
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
                constexpr bool WHOLE = C::MODE == kWgrad && !C::SPLIT && sizeof(typename C::OT) == 4;
                const bool whole = WHOLE && ep.vec == 2 && n0 + C::BN <= ep.cols;
                if constexpr (WHOLE) {
                    if (ok && whole) emit_sums<NJ>(ep, sum, m0 + lane, n0 + half * 32);
                }
#pragma unroll
                for (int jj = 0; jj < NJ; ++jj)
                    if (ok && !whole && group(jj) * 32 < C::BN) {
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
                const int64_t c = int64_t(mt) * 128 + tid;
                if (rank == 0 && nt == 0 && tid < 128 && c < ep.rows) {
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

// ---- host side ------------------------------------------------------------------------
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
    if (C::REGS && e == cudaSuccess) {             // the registers that the warpgroups share out are there
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, k_linear<C>);
        if (e == cudaSuccess && a.numRegs != 168) return cudaErrorInvalidConfiguration;
    }
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launches one configuration: splits CTAs per tile (SPLIT), else a persistent grid.
template <class C>
cudaError_t launch_cfg(const LinProblem& p, int splits, cudaStream_t st, int slabs = 1) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = prepare_kernel<C>(dev)) != cudaSuccess) return e;
    CUtensorMap ma, mb;
    if ((e = make_map(&ma, C::ROWS_M ? p.rows_op : p.cols_op, C::PL, C::A_MN ? kKb : 128)) != cudaSuccess) return e;
    if ((e = make_map(&mb, C::ROWS_M ? p.cols_op : p.rows_op, C::PL, C::B_MN ? kKb : C::BROWS)) != cudaSuccess) return e;
    const int64_t M = C::ROWS_M ? p.epi.rows : p.epi.cols, N = C::ROWS_M ? p.epi.cols : p.epi.rows;
    const int64_t mt = ceil_div(M, 128 * C::CG), nt = ceil_div(N, C::BN), kb = ceil_div(p.K, kKb);
    const int per = C::CG == 2 ? 2 : C::SPLIT ? splits : 1;
    // tile numbers, K steps and tile coordinates are 32-bit
    if (mt * nt * per > INT32_MAX / 16 || kb > INT32_MAX / 128 || M > INT32_MAX - 512 || N > INT32_MAX - 512)
        return cudaErrorInvalidValue;
    LinShape sh{int32_t(mt), int32_t(nt), int32_t(kb), splits, slabs};
    int64_t clusters = mt * nt * slabs;
    const int64_t room = sm_count(dev) / per;
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
    const float waves = float(ceil_div(tiles, room));
    if (C::SPLIT) return waves * (c.fixed + (splits > 1 ? 0.7f : 0.f) + float(ceil_div(kb, splits)) * c.kb + c.epi);
    return c.fixed + waves * float(kb) * c.kb + c.epi;
}

// The configuration with the lowest estimate.  Measured on GB300 (us, forward, bf16, rows x in
// x out; 256 x 256 pair / 256 x 128 pair / best split): 8192 x 4096 x 11008 382 / 452 / 1248;
// 2048^3 18.8 / 18.7 / 42; 333 x 2048 x 2048 - / 11 / 11; 1 x 2048 x 2048 13.3 / 9.2 / 5.8 (32
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
    float best = estimate<P256>(p, 1, dev, {6.0f, 0.275f * f, 4.5f});
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
