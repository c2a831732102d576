// linear_wgrad.cu -- dw (+)= dz^T x, the weight gradient of a linear layer, and db (+)= the
// column sums of dz.
#include "linear_kernel.cuh"

namespace fsdp {

cudaError_t launch_linear_wgrad(const LinProblem& p, cudaStream_t st) {
    if (p.planes == 3)
        return p.out_bf16 ? launch_product<kWgrad, uint16_t, 3, 0>(p, st)
                          : launch_product<kWgrad, float, 3, 2>(p, st);
    return p.out_bf16 ? launch_product<kWgrad, uint16_t, 1, 0>(p, st)
                      : launch_product<kWgrad, float, 1, 8>(p, st);
}

// ---------------------------------------------------------------------------------------
// Column sums.  A cluster of 8 CTAs owns 64 columns: CTA r adds the rows r, r + 8, ... of
// its share in fp32 (256 threads: 32 column pairs x 8 row lanes), the partial sums meet in
// CTA 0's shared memory and are added in a fixed order, so the result is the same in every
// run.
constexpr int kCsThreads = 256, kCsCols = 64, kCsRanks = 8;

template <typename T>
__device__ __forceinline__ float2 load2(const T* p, int n) {
    return make_float2(n > 0 ? load1(p) : 0.f, n > 1 ? load1(p + 1) : 0.f);
}

namespace {
template <typename T, typename OT>
__global__ void __launch_bounds__(kCsThreads)
k_colsum(const T* __restrict__ dz, int64_t rows, int64_t cols, int64_t ld, OT* db, bool accumulate) {
    __shared__ float part[kCsRanks][kCsCols];
    __shared__ float2 lanes[8][32];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t c = int64_t(blockIdx.x / kCsRanks) * kCsCols + 2 * x;
    const int n = cols - c >= 2 ? 2 : int(cols - c);
    pdl_wait();
    float2 s0 = make_float2(0.f, 0.f), s1 = s0, s2 = s0, s3 = s0;
    const int64_t step = 8 * kCsRanks;
    int64_t r = int64_t(y) * kCsRanks + rank;
    for (; r + 3 * step < rows; r += 4 * step) {
        const float2 a = load2(dz + r * ld + c, n), b = load2(dz + (r + step) * ld + c, n);
        const float2 d = load2(dz + (r + 2 * step) * ld + c, n), e = load2(dz + (r + 3 * step) * ld + c, n);
        s0.x += a.x; s0.y += a.y; s1.x += b.x; s1.y += b.y;
        s2.x += d.x; s2.y += d.y; s3.x += e.x; s3.y += e.y;
    }
    for (; r < rows; r += step) {
        const float2 a = load2(dz + r * ld + c, n);
        s0.x += a.x; s0.y += a.y;
    }
    lanes[y][x] = make_float2((s0.x + s1.x) + (s2.x + s3.x), (s0.y + s1.y) + (s2.y + s3.y));
    __syncthreads();
    if (y == 0) {
        float2 t = lanes[0][x];
        for (int k = 1; k < 8; ++k) {
            t.x += lanes[k][x].x;
            t.y += lanes[k][x].y;
        }
        const uint32_t dst = map_rank(smem_addr(&part[rank][2 * x]), 0);
        st_cluster(dst, t.x);
        st_cluster(dst + 4, t.y);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && threadIdx.x < kCsCols) {
        const int64_t cc = int64_t(blockIdx.x / kCsRanks) * kCsCols + threadIdx.x;
        if (cc < cols) {
            float t = part[0][threadIdx.x];
            for (int k = 1; k < kCsRanks; ++k) t += part[k][threadIdx.x];
            if (accumulate) t += load1(db + cc);
            store1(db + cc, t);
        }
    }
}

template <typename T, typename OT>
cudaError_t colsum(const void* dz, int64_t rows, int64_t cols, int64_t ld, void* db, bool accumulate, cudaStream_t st) {
    const int64_t groups = ceil_div(cols, kCsCols);
    if (groups > INT32_MAX / kCsRanks) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCsRanks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * kCsRanks));
    cfg.blockDim = dim3(kCsThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_colsum<T, OT>, static_cast<const T*>(dz), rows, cols, ld, static_cast<OT*>(db), accumulate);
}
}  // namespace

cudaError_t launch_colsum(const void* dz, bool dz_bf16, int64_t rows, int64_t cols, int64_t ld, void* db, bool db_bf16,
                          bool accumulate, cudaStream_t st) {
    if (dz_bf16)
        return db_bf16 ? colsum<uint16_t, uint16_t>(dz, rows, cols, ld, db, accumulate, st)
                       : colsum<uint16_t, float>(dz, rows, cols, ld, db, accumulate, st);
    return db_bf16 ? colsum<float, uint16_t>(dz, rows, cols, ld, db, accumulate, st)
                   : colsum<float, float>(dz, rows, cols, ld, db, accumulate, st);
}

cudaError_t take_wait_error_wgrad(unsigned int* flag) { return take_local_wait_error(flag); }

}  // namespace fsdp
