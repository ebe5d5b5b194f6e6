// kernels_persistent.cu -- the persistent tcgen05 GEMM (persistent.cuh) alone and
// with adapter steps, for every output type.
#include "persistent.cuh"

namespace dgb {

template <int CG, int OUT>
__global__ void __launch_bounds__(kThreads, 1) persistent_kernel(const __grid_constant__ PersistentParams p) {
    persistent_body<CG, OUT, false>(p, nullptr);
}

// The product with a tail of adapter steps after each tile's K blocks (lora.cu): rank / 16 more K = 16 instructions per
// adapter among the tile's rows.  Bound like the product by the tensor cores: 8192^3 bf16, 512-wide pair tiles, prompts of
// 12 requests with rank 64: 556 us a launch on a cool device, 2.0 PFLOP/s.  fp32 outputs: two terms of T, and the repair's
// bookkeeping beside 32 fp32 values does not fit the registers (104 bytes stored, 304 to 312 loaded a thread, once per tile
// row): 667 us a call where bf16 outputs take 638.
template <int CG, int OUT>
__global__ void __launch_bounds__(kThreads, 1) adapters_kernel(const __grid_constant__ PersistentParams p,
                                                               const __grid_constant__ LoraTail tail) {
    persistent_body<CG, OUT, true>(p, &tail);
}

// The shared-memory limit set for a kernel on each device.
template <int CG, int OUT>
static std::atomic<int> (&persistent_smem())[kMaxDevices] {
    static std::atomic<int> smem_set[kMaxDevices];
    return smem_set;
}

template <int CG, int OUT>
static cudaError_t launch_typed(const PersistentParams& p, int grid, size_t smem, cudaStream_t stream) {
    return launch_pipeline<CG>(persistent_kernel<CG, OUT>, persistent_smem<CG, OUT>(), grid, smem, stream, p);
}

template <int CG, int OUT>
static cudaError_t launch_adapters_typed(const PersistentParams& p, const LoraTail& tail, int grid, size_t smem,
                                         cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    return launch_pipeline<CG>(adapters_kernel<CG, OUT>, smem_set, grid, smem, stream, p, tail);
}

template <int CG, int OUT>
static int max_clusters_typed(size_t smem) {
    auto kern = persistent_kernel<CG, OUT>;
    if (ensure_smem_limit(kern, smem, persistent_smem<CG, OUT>()) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
    return n;
}

int persistent_max_active_clusters(int cta_group, int dtype_d, size_t smem_bytes) {
    if (cta_group == 1) {
        switch (dtype_d) {
        case GEMM_F32: return max_clusters_typed<1, GEMM_F32>(smem_bytes);
        case GEMM_BF16: return max_clusters_typed<1, GEMM_BF16>(smem_bytes);
        case GEMM_F16: return max_clusters_typed<1, GEMM_F16>(smem_bytes);
        default: return 0;
        }
    }
    switch (dtype_d) {
    case GEMM_F32: return max_clusters_typed<2, GEMM_F32>(smem_bytes);
    case GEMM_BF16: return max_clusters_typed<2, GEMM_BF16>(smem_bytes);
    case GEMM_F16: return max_clusters_typed<2, GEMM_F16>(smem_bytes);
    default: return 0;
    }
}

cudaError_t launch_persistent(const PersistentParams& p, int cta_group, int dtype_d, int grid,
                              size_t smem_bytes, cudaStream_t stream) {
    if (cta_group == 1) {
        switch (dtype_d) {
        case GEMM_F32: return launch_typed<1, GEMM_F32>(p, grid, smem_bytes, stream);
        case GEMM_BF16: return launch_typed<1, GEMM_BF16>(p, grid, smem_bytes, stream);
        case GEMM_F16: return launch_typed<1, GEMM_F16>(p, grid, smem_bytes, stream);
        default: return cudaErrorInvalidValue;
        }
    }
    switch (dtype_d) {
    case GEMM_F32: return launch_typed<2, GEMM_F32>(p, grid, smem_bytes, stream);
    case GEMM_BF16: return launch_typed<2, GEMM_BF16>(p, grid, smem_bytes, stream);
    case GEMM_F16: return launch_typed<2, GEMM_F16>(p, grid, smem_bytes, stream);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_adapters(const PersistentParams& p, const LoraTail& tail, int cta_group, int dtype_d, int grid,
                            size_t smem_bytes, cudaStream_t stream) {
    if (cta_group == 1) {
        switch (dtype_d) {
        case GEMM_F32: return launch_adapters_typed<1, GEMM_F32>(p, tail, grid, smem_bytes, stream);
        case GEMM_BF16: return launch_adapters_typed<1, GEMM_BF16>(p, tail, grid, smem_bytes, stream);
        case GEMM_F16: return launch_adapters_typed<1, GEMM_F16>(p, tail, grid, smem_bytes, stream);
        default: return cudaErrorInvalidValue;
        }
    }
    switch (dtype_d) {
    case GEMM_F32: return launch_adapters_typed<2, GEMM_F32>(p, tail, grid, smem_bytes, stream);
    case GEMM_BF16: return launch_adapters_typed<2, GEMM_BF16>(p, tail, grid, smem_bytes, stream);
    case GEMM_F16: return launch_adapters_typed<2, GEMM_F16>(p, tail, grid, smem_bytes, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dgb
