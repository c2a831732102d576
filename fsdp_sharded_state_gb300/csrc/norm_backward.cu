// norm_backward.cu -- the gradients of a layer norm.
//
// With h = (x - mean) * rstd and g = dy * weight:
//     dx = residual + rstd * (g - mean over the row of g - h * mean over the row of g h)
//     dw (+)= sum over rows of dy h;   db (+)= sum over rows of dy
//
// Bound by HBM: x, dy and the residual read, dx written once.  dw and db cost no second pass: a
// thread keeps its columns of every row that its CTA works on, adds them up in fp32 registers,
// and leaves one row of partial sums per CTA, which k_norm_join adds up in a fixed order.
//
// bf16 with a residual, one GB300, without and with the sums: 16384 x 4096 77 and 84 us (the copy rate, 79,
// and the join), 65536 x 256 24 and 28 (0.7: neither HBM nor the issue of instructions, 47 %, is full), 4096 x 16384 84 and 95; fp32
// 8192 x 4096 79 and 85.
#include "norm_rows.cuh"

namespace fsdp {
namespace {

struct BackwardArgs {
    const void* x;
    int64_t ldx;
    const void* dy;
    int64_t lddy;
    const void* weight;
    const void* residual;
    int64_t ldr;
    const float* mean;
    const float* rstd;
    void* dx;
    int64_t lddx;
    float* partial;                 // [2][groups][pitch], or NULL
    int64_t pitch, rows;
    int32_t cols, ctas, stages, block;
    uint64_t wait_ns;
};

// Columns of a row of partial sums.
__host__ __device__ inline int64_t partial_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

// CTAs of an SM: threads of up to 128 registers (168 in CTAs of 384).
template <class C>
constexpr int kBackwardCtas = 512 / C::THREADS;

template <class C>
__global__ void __launch_bounds__(C::THREADS, kBackwardCtas<C>)
k_norm_backward(const __grid_constant__ BackwardArgs a) {
    using T = typename C::T;
    using Sums = RowSum<C, 2>;
    extern __shared__ __align__(128) unsigned char smem_raw[];   // the ring; at the end a row of sums per group
    __shared__ __align__(16) float sums[C::GW > 1 ? Sums::FLOATS * C::SIDE : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t = C::GW == 1 ? lane % C::L : tid % C::G, group = warp / C::GW;
    const int rank = C::CLUSTER ? int(cluster_rank()) : 0, first = rank * C::COLS;
    const int part = blockIdx.x / a.ctas, parts = gridDim.x / a.ctas;
    const bool res = a.residual != nullptr;
    const uint32_t rows = uint32_t(a.rows), row0 = part * uint32_t(C::SIDE * a.block);
    RowRing<C, 3> ring(smem_raw, first, a.cols, a.stages, a.block, rows, parts * uint32_t(C::SIDE * a.block), a.wait_ns);
    ring.matrix(0, a.x, a.ldx, first, row0);
    ring.matrix(1, a.dy, a.lddy, first, row0);
    ring.matrix(2, a.residual, a.ldr, first, row0);
    if (tid == 0) ring.init();
    if constexpr (C::CLUSTER) {                  // no CTA writes to another that has not started
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    pdl_wait();
    if (C::SIDE == 1 ? tid == 0 : warp == 0) ring.begin(row0, lane);
    pair w[C::P], dw[C::P], db[C::P];
    norm_vector<C>(static_cast<const T*>(a.weight), a.cols, first, t, 1.f, w);
#pragma unroll
    for (int i = 0; i < C::P; ++i) dw[i] = db[i] = 0;
    Sums sum{sums, ring.sums(0), a.wait_ns};
    const bool full = __all_sync(0xffffffffu, norm_full<C>(a.cols, first, t));
    const float over_n = 1.f / float(a.cols);
    // of the group's first row of the stage: its place in it and in dx
    const int block = C::GW == 1 ? a.block : 1;
    const int j1 = group * block + (C::GW == 1 ? lane / C::L : 0);
    uint32_t mine = row0 + j1;
    T* py = static_cast<T*>(a.dx) + mine * a.lddx;
    const int64_t y_step = ring.step * a.lddx, y_side = (32 / C::L) * a.lddx;
    // mean and rstd are read a stage ahead: of the group's l-th row by lane l where that is a warp
    float next_mean = 0.f, next_rstd = 0.f;
    auto read_ahead = [&](uint32_t row) {
        row += group * block + (C::GW == 1 ? lane : 0);
        if ((C::GW > 1 || lane < block) && row < rows) {
            next_mean = a.mean[row];
            next_rstd = a.rstd[row];
        }
    };
    read_ahead(row0);
    // the threads of a CTA, or of a cluster, leave the loop together
    for (uint32_t row = row0; row < rows; row += ring.step, mine += ring.step, py += y_step) {
        const float row_mean = next_mean, row_rstd = next_rstd;
        read_ahead(row + ring.step);
        ring.wait();
        T* y = py;
        for (int j0 = 0; j0 < block; j0 += C::GW == 1 ? 32 / C::L : 1, y += y_side) {
            const bool have = mine + j0 < rows;
            pair h[C::P], g[C::P], add[C::P];
            float v[2] = {0.f, 0.f}, mean = row_mean, rstd = row_rstd;
            if constexpr (C::GW == 1) {
                mean = __shfl_sync(0xffffffffu, row_mean, j0 + lane / C::L);
                rstd = __shfl_sync(0xffffffffu, row_rstd, j0 + lane / C::L);
            }
            if (have) {
                norm_load<C>(ring.row_of(j1 + j0, 0), a.cols, first, t, full, h);
                norm_load<C>(ring.row_of(j1 + j0, 1), a.cols, first, t, full, g);
                if (C::GW > 1 && res) norm_load<C>(ring.row_of(j1 + j0, 2), a.cols, first, t, full, add);
                const pair m = pair_of(-mean, -mean), r = pair_of(rstd, rstd);
#pragma unroll
                for (int i = 0; i < C::P; ++i) h[i] = mul2(add2(h[i], m), r);
                if (!full) norm_trim<C>(a.cols, first, t, h);
                pair p = 0, q = 0;
#pragma unroll
                for (int i = 0; i < C::P; ++i) {
                    dw[i] = fma2(g[i], h[i], dw[i]);
                    db[i] = add2(db[i], g[i]);
                    g[i] = mul2(g[i], w[i]);
                    p = add2(p, g[i]);
                    q = fma2(g[i], h[i], q);
                }
                v[0] = both(p);
                v[1] = both(q);
            }
            sum(v, warp, lane, a.ctas);
            if (C::GW > 1) {                     // every thread of the group has read its row
                if (C::SIDE == 1 ? tid == 0 : warp % C::GW == 0) ring.release(row, lane);
                ring.next();
            }
            if (!have) continue;
            const float c0 = -v[0] * over_n, c1 = -v[1] * over_n;
            const pair m0 = pair_of(c0, c0), m1 = pair_of(c1, c1), r = pair_of(rstd, rstd);
            if (C::GW == 1 && C::VEC) {          // the residual a chunk at a time: as a whole its registers spill, and 65536 x 256 takes 33 us
                const uint32_t from = ring.row_of(j1 + j0, 2);
#pragma unroll
                for (int c = 0; c < C::P; c += C::W / 2) {
                    pair add4[C::W / 2];
                    const int col = norm_col<C>(0, t, 2 * c);
                    if (res) {
                        smem_get16(full || col < a.cols ? from + uint32_t(col) * uint32_t(sizeof(T)) : from, add4, static_cast<const T*>(nullptr));
                    } else {
#pragma unroll
                        for (int i = 0; i < C::W / 2; ++i) add4[i] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < C::W / 2; ++i) g[c + i] = fma2(fma2(h[c + i], m1, add2(g[c + i], m0)), r, add4[i]);
                }
            } else if (res) {
                if (C::GW == 1) norm_load<C>(ring.row_of(j1 + j0, 2), a.cols, first, t, full, add);
#pragma unroll
                for (int i = 0; i < C::P; ++i) g[i] = fma2(fma2(h[i], m1, add2(g[i], m0)), r, add[i]);
            } else {
#pragma unroll
                for (int i = 0; i < C::P; ++i) g[i] = mul2(fma2(h[i], m1, add2(g[i], m0)), r);
            }
            norm_store<C>(y, a.cols, first, t, full, g);
        }
        if (C::GW == 1) {
            __syncwarp();                        // every lane has read the warp's rows
            ring.release(row, lane);
            ring.next();
        }
    }
    ring.leave(C::CLUSTER ? sum.wait_ns : 1);
    if (!a.partial) return;
    float* const out_w = a.partial + part * a.pitch;
    float* const out_b = out_w + parts * a.pitch;
    if constexpr (C::SIDE > 1) {
        // the rows of a warp, then the groups of the CTA, in order
        float* const smem = reinterpret_cast<float*>(smem_raw);
#pragma unroll
        for (int o = 16; o >= C::L; o >>= 1)
#pragma unroll
            for (int i = 0; i < C::P; ++i) {
                dw[i] = add2(dw[i], __shfl_xor_sync(0xffffffffu, dw[i], o));
                db[i] = add2(db[i], __shfl_xor_sync(0xffffffffu, db[i], o));
            }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            if (C::GW > 1 || lane < C::L) {
#pragma unroll
                for (int e = 0; e < C::E; e += 2) {
                    const float2 f = split(which ? db[e / 2] : dw[e / 2]);
                    smem[warp / C::GW * C::COLS + norm_col<C>(0, t, e)] = f.x;
                    smem[warp / C::GW * C::COLS + norm_col<C>(0, t, e + 1)] = f.y;
                }
            }
            __syncthreads();
            for (int c = tid; c < a.cols; c += C::THREADS) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < C::SIDE; ++k) v += smem[k * C::COLS + c];
                (which ? out_b : out_w)[c] = v;
            }
        }
    } else {
        if (C::VEC) {                            // whole sectors: element by element they took 10 us of 16384 x 4096
#pragma unroll
            for (int e = 0; e < C::E; e += 4) {
                const int c = norm_col<C>(first, t, e);
                if (c >= a.cols) continue;
                const float2 f = split(dw[e / 2]), g = split(dw[e / 2 + 1]), u = split(db[e / 2]), v = split(db[e / 2 + 1]);
                st4(out_w + c, make_float4(f.x, f.y, g.x, g.y));
                st4(out_b + c, make_float4(u.x, u.y, v.x, v.y));
            }
        } else {
#pragma unroll
            for (int e = 0; e < C::E; ++e) {
                const int c = norm_col<C>(first, t, e);
                if (c < a.cols) {
                    const float2 f = split(dw[e / 2]), g = split(db[e / 2]);
                    out_w[c] = e & 1 ? f.y : f.x;
                    out_b[c] = e & 1 ? g.y : g.x;
                }
            }
        }
    }
}

// out[c] (+)= the sum over p of part[p][c], for dw and (blockIdx.y = 1) db.  A block takes 32
// columns; its kJoinWarps warps every kJoinWarps-th row each, and then warp 0 adds the warps'
// sums up in order.
constexpr int kJoinWarps = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps)
k_norm_join(const float* part, int parts, int64_t pitch, int cols, T* dw, T* db, bool accumulate) {
    __shared__ float sums[kJoinWarps][32];
    pdl_wait();
    T* const out = blockIdx.y ? db : dw;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* const src = part + (blockIdx.y ? parts * pitch : 0);
    float v = 0.f;
    if (out && c < cols) {
#pragma unroll 10
        for (int p = warp; p < parts; p += kJoinWarps) v += src[p * pitch + c];
    }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && out && c < cols) {
        v = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) v += sums[k][lane];
        if (accumulate) v += norm_get(out + c);
        norm_put(out + c, v);
    }
}

// CTAs (or clusters) that work through the rows, each with a row of partial sums: as many as
// fit the 152 SMs at once, fewer where there are few rows.
template <class C>
int64_t backward_groups(int64_t rows, int64_t cols) {
    const int64_t each = ring_shape<C>(3, cols, kBackwardCtas<C>).block * C::SIDE;
    const int64_t want = (rows + each - 1) / each, room = 152 * kBackwardCtas<C> / norm_ctas<C>(cols);
    return want < room ? want : room;
}

template <class C>
cudaError_t launch_as(const NormProblem& p, cudaStream_t st) {
    const int ctas = norm_ctas<C>(p.cols);
    const int64_t groups = backward_groups<C>(p.rows, p.cols), pitch = partial_pitch(p.cols);
    const bool sums = p.dw || p.db;
    cudaError_t e = cudaSuccess;
    if (p.rows > 0) {
        static std::atomic<uint64_t> prepared{0};
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess || (e = norm_prepare(k_norm_backward<C>, prepared, dev)) != cudaSuccess) return e;
        const RingShape ring = ring_shape<C>(3, p.cols, kBackwardCtas<C>);
        const size_t last = C::SIDE > 1 ? size_t(C::SIDE) * C::COLS * 4 : 0;
        const BackwardArgs a{p.x, p.ldx, p.dy, p.lddy, p.weight, p.residual, p.ldr, p.mean, p.rstd, p.y, p.ldy,
                             sums ? p.partial : nullptr, pitch, p.rows, int32_t(p.cols), ctas, ring.stages, ring.block, detail::kWaitNs};
        e = norm_launch(k_norm_backward<C>, int(groups), ctas, C::THREADS, ring.bytes > last ? ring.bytes : last, st, a);
    }
    if (e != cudaSuccess || !sums || (p.rows == 0 && p.accumulate)) return e;
    const dim3 grid(unsigned((p.cols + 31) / 32), 2);
    if (p.grad_bf16)
        return launch(k_norm_join<uint16_t>, grid, dim3(32 * kJoinWarps), 0, st, static_cast<const float*>(p.partial), int(groups), pitch,
                      int(p.cols), static_cast<uint16_t*>(p.dw), static_cast<uint16_t*>(p.db), p.accumulate);
    return launch(k_norm_join<float>, grid, dim3(32 * kJoinWarps), 0, st, static_cast<const float*>(p.partial), int(groups), pitch,
                  int(p.cols), static_cast<float*>(p.dw), static_cast<float*>(p.db), p.accumulate);
}

}  // namespace

int64_t norm_partial_floats(int64_t rows, int64_t cols) {
    int64_t groups = 0;
    auto most = [&](auto c) {
        const int64_t g = backward_groups<decltype(c)>(rows, cols);
        if (g > groups) groups = g;
        return cudaSuccess;
    };
    norm_dispatch_backward<float, true>(cols, most);
    norm_dispatch_backward<uint16_t, true>(cols, most);
    return 2 * groups * partial_pitch(cols);
}

cudaError_t take_wait_error_norm_backward(unsigned int* flag) { return take_norm_wait_error(flag); }

cudaError_t launch_norm_backward(const NormProblem& p, cudaStream_t st) {
    auto go = [&](auto c) { return launch_as<decltype(c)>(p, st); };
    if (p.bf16) return p.vec ? norm_dispatch_backward<uint16_t, true>(p.cols, go) : norm_dispatch_backward<uint16_t, false>(p.cols, go);
    return p.vec ? norm_dispatch_backward<float, true>(p.cols, go) : norm_dispatch_backward<float, false>(p.cols, go);
}

}  // namespace fsdp
