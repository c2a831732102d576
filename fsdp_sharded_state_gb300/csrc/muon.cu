// muon.cu -- the ZeRO-1 Muon step: momentum of the mean gradient, Newton-Schulz steps, weight
// decay and the broadcast of the new weights (extern "C" entry points and the two passes around the
// products).
//
// The first pass reads the N gradient replicas and the momentum and writes the momentum, the
// update (4 bytes an element, into the workspace) and its sum of squares; the last one reads the
// orthogonalised update and the weights and writes these and N replicas.  Both are bound by HBM; each
// tensor's rows in the shard and in the full layout line up mod 8, so every access but a tensor's
// first and last is a 16-byte vector.  The division by the norm waits for all squares, so it is done where
// the products' first operand is formed.
#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "device_ops.cuh"
#include "internal.hpp"
#include "ns.hpp"

namespace fsdp {
namespace {

constexpr int kMuonThreads = 256;

struct MuonJobs {
    int64_t shard[kNsMaxBatch];     // element in the [N][stride] rows
    int64_t full[kNsMaxBatch];      // element in the full layout, congruent mod 8
    float step[kNsMaxBatch];        // lr * scale
    int32_t owner[kNsMaxBatch];
    int64_t numel;
    float* update;                  // matrix i at update + i pitch + (shard[i] mod 8)
    int64_t pitch;
    int32_t N;
    float nf;                       // N
};
struct MuonReplicas {
    void* p[kMaxRanks];
};

__device__ __forceinline__ float muon_block_sum(float v) {
    __shared__ float part[kMuonThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.f;
        for (int k = 0; k < kMuonThreads / 32; ++k) v += part[k];
    }
    return v;
}

// The sum of the N replicas at 8 neighbours, in rank order, two loads at once: what a thread holds
// for more of them costs threads (a batch of eight: 4096 x 11008, N = 2, 154 us; two: 110, of 106 at HBM's rate).
template <typename GT>
__device__ __forceinline__ void replicas8(const GradPtrs& gp, int N, int64_t f, float (&sum)[8]) {
    using IO = GradIO<GT>;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = 0.f;
    for (int q = 0; q < N; q += 2) {
        const bool two = q + 1 < N;
        const typename IO::Vec a = IO::load(gp.p[q], f), b = two ? IO::load(gp.p[q + 1], f) : a;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sum[k] = __fadd_rn(sum[k], IO::elem(a, a, k));
            if (two) sum[k] = __fadd_rn(sum[k], IO::elem(b, b, k));
        }
    }
}

// m = beta m + (1 - beta) g, g the mean of the replicas; the update is m, or (nesterov)
// beta m + (1 - beta) g of the new m.
template <typename GT>
__global__ void __launch_bounds__(kMuonThreads)
k_muon_momentum(const __grid_constant__ MuonJobs jobs, const __grid_constant__ GradPtrs gp, float* momentum, float beta, float om,
                int nesterov, float* partial) {
    pdl_wait();
    pdl_trigger();
    const int mat = blockIdx.y;
    const int64_t lo = jobs.shard[mat], hi = lo + jobs.numel, delta = jobs.full[mat] - lo;
    float* const u = jobs.update + mat * jobs.pitch + (lo & 7) - lo;
    float total = 0.f, lost = 0.f;
    auto one = [&](float g, float& m) {
        const float gg = __fmul_rn(om, mean_div(g, jobs.nf));
        m = __fmaf_rn(beta, m, gg);
        return nesterov ? __fmaf_rn(beta, m, gg) : m;
    };
    const int64_t step = int64_t(gridDim.x) * kMuonThreads * 8;
    int64_t e0 = (lo & ~int64_t(7)) + (int64_t(blockIdx.x) * kMuonThreads + threadIdx.x) * 8;
    auto finish = [&](int64_t e, float (&g)[8], const float4& a, const float4& b) {
        float m[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            g[k] = one(g[k], m[k]);
            s = __fmaf_rn(g[k], g[k], s);
        }
        st4(momentum + e, make_float4(m[0], m[1], m[2], m[3]));
        st4(momentum + e + 4, make_float4(m[4], m[5], m[6], m[7]));
        st4(u + e, make_float4(g[0], g[1], g[2], g[3]));
        st4(u + e + 4, make_float4(g[4], g[5], g[6], g[7]));
        add_carefully(s, total, lost);
    };
    for (; e0 < hi; e0 += step) {
        if (e0 >= lo && e0 + 8 <= hi) {
            const float4 a = ld4(momentum + e0), b = ld4(momentum + e0 + 4);
            float g[8];
            replicas8<GT>(gp, jobs.N, e0 + delta, g);
            finish(e0, g, a, b);
        } else {
            float s = 0.f;
            for (int64_t e = e0 > lo ? e0 : lo; e < (e0 + 8 < hi ? e0 + 8 : hi); ++e) {
                float m = momentum[e];
                const float v = one(reduce1<GT>(gp, jobs.N, e + delta), m);
                momentum[e] = m;
                u[e] = v;
                s = __fmaf_rn(v, v, s);
            }
            add_carefully(s, total, lost);
        }
    }
    total = muon_block_sum(total);
    if (threadIdx.x == 0) partial[mat * gridDim.x + blockIdx.x] = total;
}

// w = decay w - step O, into the master rows and every replica.
template <bool MASTER>
__global__ void __launch_bounds__(kMuonThreads)
k_muon_apply(const __grid_constant__ MuonJobs jobs, float* master, const __grid_constant__ MuonReplicas out, float decay) {
    pdl_wait();
    const int mat = blockIdx.y;
    const int64_t lo = jobs.shard[mat], hi = lo + jobs.numel, delta = jobs.full[mat] - lo;
    const float* const o = jobs.update + mat * jobs.pitch + (lo & 7) - lo;
    const float step = jobs.step[mat];
    const float* const own = static_cast<const float*>(out.p[jobs.owner[mat]]);
    for (int64_t e0 = (lo & ~int64_t(7)) + (int64_t(blockIdx.x) * kMuonThreads + threadIdx.x) * 8; e0 < hi;
         e0 += int64_t(gridDim.x) * kMuonThreads * 8) {
        if (e0 >= lo && e0 + 8 <= hi) {
            const float* const src = MASTER ? master + e0 : own + e0 + delta;
            const float4 a = ld4(src), b = ld4(src + 4), c = ld4(o + e0), d = ld4(o + e0 + 4);
            float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const float x[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = __fmaf_rn(-step, x[k], __fmul_rn(w[k], decay));
            if constexpr (MASTER) {
                st4(master + e0, make_float4(w[0], w[1], w[2], w[3]));
                st4(master + e0 + 4, make_float4(w[4], w[5], w[6], w[7]));
                const uint4 q = make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7]));
                for (int r = 0; r < jobs.N; ++r) stu4(static_cast<uint16_t*>(out.p[r]) + e0 + delta, q);
            } else {
                for (int r = 0; r < jobs.N; ++r) {
                    float* const p = static_cast<float*>(out.p[r]) + e0 + delta;
                    st4(p, make_float4(w[0], w[1], w[2], w[3]));
                    st4(p + 4, make_float4(w[4], w[5], w[6], w[7]));
                }
            }
        } else {
            for (int64_t e = e0 > lo ? e0 : lo; e < (e0 + 8 < hi ? e0 + 8 : hi); ++e) {
                const float w = __fmaf_rn(-step, o[e], __fmul_rn(MASTER ? master[e] : own[e + delta], decay));
                if (MASTER) master[e] = w;
                for (int r = 0; r < jobs.N; ++r) {
                    if (MASTER) static_cast<uint16_t*>(out.p[r])[e + delta] = to_bf16(w);
                    else static_cast<float*>(out.p[r])[e + delta] = w;
                }
            }
        }
    }
}

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Tensors of one pair of sides, in the caller's order.
struct Group {
    int64_t m, n;
    std::vector<int32_t> tensors;
};

// Workspace of a group: the products', then the updates.
struct GroupWork {
    NsWork ns;
    int64_t update, pitch, end;     // bytes, floats, bytes
};
GroupWork group_work(const Group& g) {
    GroupWork w;
    w.ns = ns_work(g.m, g.n, int64_t(g.tensors.size()));
    w.pitch = round_up(g.m * g.n + 8, 64);
    w.update = round_up(w.ns.end, 256);
    w.end = w.update + w.ns.chunk * w.pitch * 4;
    return w;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::detail;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxElems = int64_t(1) << 34;

// The groups of a list of tensors, checked.
int make_groups(const fsdp_layout* L, int32_t n, const int32_t* ids, std::vector<Group>* out) {
    if (!L || n < 0 || (n > 0 && !ids)) return FSDP_EINVAL;
    if (L->mode != FSDP_ZERO1) return FSDP_EINVAL;
    std::vector<bool> seen(size_t(L->T), false);
    for (int32_t i = 0; i < n; ++i) {
        const int32_t t = ids[i];
        if (t < 0 || t >= L->T || seen[size_t(t)]) return FSDP_EINVAL;
        seen[size_t(t)] = true;
        const int64_t r = L->d0[size_t(t)], c = L->inner[size_t(t)];
        if (r < 1 || c < 2) return FSDP_ESHAPE;
        if (r > kMaxDim || c > kMaxDim || round_up(r, 256) * round_up(c, 256) > kMaxElems) return FSDP_EOVERFLOW;
        const int64_t m = std::min(r, c), k = std::max(r, c);
        auto at = std::find_if(out->begin(), out->end(), [&](const Group& g) { return g.m == m && g.n == k; });
        if (at == out->end()) {
            out->push_back(Group{m, k, {}});
            at = out->end() - 1;
        }
        at->tensors.push_back(t);
    }
    return FSDP_OK;
}

// And the workspace they need; what the lists cannot be allocated for is FSDP_ENOMEM.
int groups_of(const fsdp_layout* L, int32_t n, const int32_t* ids, std::vector<Group>* out, int64_t* bytes) {
    try {
        const int rc = make_groups(L, n, ids, out);
        if (rc) return rc;
    } catch (const std::exception&) {
        return FSDP_ENOMEM;
    }
    *bytes = 0;
    for (const Group& g : *out) *bytes = std::max(*bytes, group_work(g).end);
    return FSDP_OK;
}

int check_muon(const fsdp_muon_hparams* hp) {
    if (!hp) return FSDP_EINVAL;
    if (!std::isfinite(hp->lr) || hp->lr < 0.f || !std::isfinite(hp->weight_decay) || hp->weight_decay < 0.f) return FSDP_EINVAL;
    if (!(hp->momentum >= 0.f) || !(hp->momentum < 1.f)) return FSDP_EINVAL;
    if (!(hp->eps >= kNsLeastEps) || !std::isfinite(hp->eps)) return FSDP_EINVAL;
    if (hp->steps < 1 || hp->steps > kNsMaxSteps) return FSDP_EINVAL;
    if (hp->scale < FSDP_MUON_SCALE_NONE || hp->scale > FSDP_MUON_SCALE_RMS) return FSDP_EINVAL;
    return FSDP_OK;
}

double scale_for(int32_t kind, int64_t rows, int64_t cols) {
    if (kind == FSDP_MUON_SCALE_SHAPE) return std::sqrt(std::max(1.0, double(rows) / double(cols)));
    if (kind == FSDP_MUON_SCALE_RMS) return 0.2 * std::sqrt(double(std::max(rows, cols)));
    return 1.0;
}

}  // namespace

extern "C" {

size_t fsdp_zero1_muon_workspace_bytes(const fsdp_layout* L, int32_t n_tensors, const int32_t* tensors) {
    std::vector<Group> groups;
    int64_t bytes = 0;
    if (groups_of(L, n_tensors, tensors, &groups, &bytes)) return 0;
    return size_t(bytes);
}

int fsdp_zero1_muon_broadcast(const fsdp_layout* L, int32_t n_tensors, const int32_t* tensors, const void* const* grads,
                              int32_t grad_dtype, float* master, float* momentum, void* const* param_replicas, int32_t param_dtype,
                              const fsdp_muon_hparams* hp, const float* coeffs, void* workspace, size_t workspace_bytes,
                              fsdp_stream_t stream) {
    NvtxRange nvtx_range("fsdp_zero1_muon_broadcast");
    std::vector<Group> groups;
    int64_t need = 0;
    int rc = groups_of(L, n_tensors, tensors, &groups, &need);
    if (rc) return rc;
    if (grad_dtype != FSDP_F32 && grad_dtype != FSDP_BF16) return FSDP_EDTYPE;
    if (param_dtype != FSDP_F32 && param_dtype != FSDP_BF16) return FSDP_EDTYPE;
    if ((param_dtype == FSDP_BF16) != (master != nullptr)) return FSDP_EINVAL;   // bf16 replicas need a master
    if (!grads || !param_replicas) return FSDP_EINVAL;
    for (int32_t q = 0; q < L->N; ++q)
        if ((rc = check_ptr(grads[q])) || (rc = check_ptr(param_replicas[q]))) return rc;
    if ((rc = check_ptr(momentum))) return rc;
    if (master && !aligned16(master)) return FSDP_EALIGN;
    if ((rc = check_muon(hp))) return rc;
    NsScales sc;
    if (!ns_scales(coeffs, hp->steps, &sc)) return FSDP_EINVAL;
    if (need > 0 && (!workspace || workspace_bytes < size_t(need))) return FSDP_EINVAL;
    if (workspace && !aligned16(workspace)) return FSDP_EALIGN;
    GradPtrs gp{};
    MuonReplicas out{};
    for (int32_t q = 0; q < L->N; ++q) {
        gp.p[q] = grads[q];
        out.p[q] = param_replicas[q];
    }
    const float decay = float(1.0 - double(hp->lr) * double(hp->weight_decay)), om = float(1.0 - double(hp->momentum));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    for (const Group& g : groups) {
        const GroupWork w = group_work(g);
        const int total = int(g.tensors.size());
        for (int first = 0; first < total; first += w.ns.chunk) {
            const int n = std::min(w.ns.chunk, total - first);
            MuonJobs jobs = {};
            jobs.numel = g.m * g.n;
            jobs.update = reinterpret_cast<float*>(ws + w.update);
            jobs.pitch = w.pitch;
            jobs.N = L->N;
            jobs.nf = float(L->N);
            NsMatrices o = {};
            for (int i = 0; i < n; ++i) {
                const size_t t = size_t(g.tensors[size_t(first + i)]);
                const int64_t rows = L->d0[t], cols = L->inner[t];
                jobs.owner[i] = L->owner[t];
                jobs.shard[i] = L->owner[t] * L->stride + L->t_shard_off[t];
                jobs.full[i] = L->t_full_off[t];
                jobs.step[i] = float(double(hp->lr) * scale_for(hp->scale, rows, cols));
                o.p[i] = jobs.update + i * w.pitch + (jobs.shard[i] & 7);
                o.ld[i] = cols;
                if (rows > cols) o.tall |= uint64_t(1) << i;
            }
            const int parts = ns_parts(jobs.numel);
            float* const partial = reinterpret_cast<float*>(ws + w.ns.partial);
            const dim3 grid(static_cast<unsigned>(parts), static_cast<unsigned>(n)), block(kMuonThreads);
            cudaError_t e = grad_dtype == FSDP_BF16
                                ? launch(k_muon_momentum<uint16_t>, grid, block, 0, st, jobs, gp, momentum, hp->momentum, om, hp->nesterov, partial)
                                : launch(k_muon_momentum<float>, grid, block, 0, st, jobs, gp, momentum, hp->momentum, om, hp->nesterov, partial);
            if (e != cudaSuccess) return cuda_fail(e, "k_muon_momentum launch");
            e = ns_run(w.ns, ws, n, o, o, parts, hp->eps, coeffs, hp->steps, sc, true, st);
            if (e != cudaSuccess) return cuda_fail(e, "k_ns launch");
            e = master ? launch(k_muon_apply<true>, grid, block, 0, st, jobs, master, out, decay)
                       : launch(k_muon_apply<false>, grid, block, 0, st, jobs, master, out, decay);
            if (e != cudaSuccess) return cuda_fail(e, "k_muon_apply launch");
        }
    }
    return FSDP_OK;
}

}  // extern "C"
