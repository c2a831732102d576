// linear_epilogue.cuh -- what happens to an accumulator of a linear layer's product before its
// one rounding: bias, activation or its derivative, dropout, residual or accumulation; and the
// column sums of dz.  Device code of linear_kernel.cuh.
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
// derivative's.  gelu is then within 2.6e-7 (erff's form within 1.6e-7): relative to its own value
// 6e-5 in [-3, -2] and 9e-4 in [-4, -3], below bf16's rounding; further down both forms take Phi's
// value from a difference of numbers near 1/2 and lose it (5 % at -5).  A tile of 256 x 256 leaves the epilogue 16,000 clocks beside the products of
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
// columns, STEP apart from col0 on, while they lie wholly inside the matrix, `most` of them, and
// returns how many; a unit's two halves are read (residual, pre-activation) while the unit before it is
// computed.  dcol: the generator's column products of the units' columns, in shared memory;
// dr: the lane's row's.
template <int MODE, int EP, bool ALIGNED>
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
    __device__ __forceinline__ void begin(const LinEpi& ep, int64_t row, int64_t col0, int most) {
        in = row < ep.rows;
        const int64_t left = ep.cols - col0;
        units = left < 32 ? 0 : (left - 32) / STEP + 1 < most ? int((left - 32) / STEP + 1) : most;
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
// columns col0 + 64 u on.  An accumulator's old values are added last and once: sums that started
// from them were rounded at the accumulator's magnitude with every chunk, and 32 chunks of 2^-26
// each left an accumulator of 1 as it was.  Its lines are brought to L2 while the first products run
// (2048^3 bf16, one call after another on the same operands: 20.2 us, 17.7 where nothing is added).
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
__device__ __forceinline__ void prefetch_sums(const LinEpi& ep, int64_t row, int64_t col0) {
    if (row >= ep.rows) return;
    const float* const in = static_cast<const float*>(ep.out) + row * ep.ldo + col0;
#pragma unroll
    for (int u = 0; u < NU; ++u) {               // 128 bytes, on two lines where rows are not aligned to one
        asm volatile("prefetch.global.L2 [%0];" ::"l"(in + 64 * u) : "memory");
        asm volatile("prefetch.global.L2 [%0];" ::"l"(in + 64 * u + 31) : "memory");
    }
}
template <int NU>
__device__ __forceinline__ void emit_sums(const LinEpi& ep, const float (&sum)[NU][32], int64_t row, int64_t col0) {
    if (row >= ep.rows) return;
    float* const out = static_cast<float*>(ep.out) + row * ep.ldo + col0;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        float* const p = out + 64 * u;
        Raw8f r[4];
        if (ep.accumulate) {
#pragma unroll
            for (int g = 0; g < 4; ++g) load_8f(p + 8 * g, r[g]);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[g].v[e] += sum[u][8 * g + e];
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[g].v[e] = sum[u][8 * g + e];
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) store_8f(p + 8 * g, r[g]);
    }
}

// ---- column sums of dz (wgrad's db) ---------------------------------------------------
// 16 to 128 columns of every second group of rows of dz added up straight from memory, which the
// tiles' own copies bring into L2.  (Added up from the shared-memory stages they held each of
// them back from its next load by more than the ring of stages covers: 16384 x 2048 x 2048 took
// 111 us against 78 without db.)  The tiles of a row of tiles share out its columns; with their
// rows shared out instead, a launch of 3 us had to join the sums.  Lane l holds columns
// E (l mod L) on, L lanes to a row.  Loads are 16 bytes wherever rows start at multiples of 16,
// ragged ends included: with the last columns' tile read by single elements, 4096 x 777 x 1001
// took 110 us instead of 25.
template <typename T>
struct RowSum {
    static constexpr int E = 16 / sizeof(T), B = 16;             // elements of a load; loads in flight
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
    // Columns col on, L lanes to a row, of the groups of 32 / L rows, every second from the half-th on.
    __device__ __forceinline__ void add(const T* dz, int64_t ld, int half, int64_t rows, int64_t col, int64_t cols, bool vec, int L,
                                        int lane) {
        const int64_t c = col + (lane & (L - 1)) * E;
        const int every = 64 / L, first = (half * 32 + lane) / L;
        int64_t r = first;
        if (c >= cols) return;
        const T* p = dz + r * ld + c;
        const int64_t step = every * ld;
        if (vec) {
            // rows start at multiples of 16 bytes, so a row's last load ends before the next row;
            // what is left of the very last row is added below
            const int64_t end = c + E <= cols ? rows : rows - 1;
#pragma unroll 1
            while (r < end) {
                uint4 q[B];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    q[i] = r < end ? ldu4(p) : make_uint4(0, 0, 0, 0);
                    r += every;
                    p += step;
                }
#pragma unroll
                for (int i = 0; i < B; i += 4) {
                    float x[4][E];
#pragma unroll
                    for (int k = 0; k < 4; ++k) wide(q[i + k], x[k]);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] += (x[0][e] + x[1][e]) + (x[2][e] + x[3][e]);
                }
            }
            if (end < rows && (rows - 1) % every == first) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] += c + e < cols ? load1(dz + (rows - 1) * ld + c + e) : 0.f;
            }
        } else {                                             // any alignment (fp32 only)
#pragma unroll 1
            while (r < rows) {
                float x[8][E];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
#pragma unroll
                    for (int e = 0; e < E; ++e) x[k][e] = r < rows && c + e < cols ? load1(p + e) : 0.f;
                    r += every;
                    p += step;
                }
#pragma unroll
                for (int e = 0; e < E; ++e)
                    v[e] += ((x[0][e] + x[1][e]) + (x[2][e] + x[3][e])) + ((x[4][e] + x[5][e]) + (x[6][e] + x[7][e]));
            }
        }
    }
    // Lane l < L: the sums of its columns over the warp.
    __device__ __forceinline__ void join(int L) {
        for (int m = L; m < 32; m <<= 1) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], m);
        }
    }
};

}  // namespace
}  // namespace fsdp
