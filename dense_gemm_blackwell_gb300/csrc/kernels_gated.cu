// kernels_gated.cu -- the persistent kernel (persistent.cuh) for a gated pair of
// projections, act(X Wg^T) * (X Wu^T): the B rows of a tile are gates and ups of
// the same output columns, so both products run as one and meet in the epilogue.
#include "persistent.cuh"

namespace dgb {

template <int CG, int OUT>
__global__ void __launch_bounds__(kThreads, 1) gated_kernel(const __grid_constant__ PersistentParams p,
                                                            const __grid_constant__ GatedTail gated) {
    persistent_body<CG, OUT, false, true>(p, nullptr, &gated);
}

template <int CG, int OUT>
static cudaError_t launch_gated_typed(const PersistentParams& p, const GatedTail& q, int grid, size_t smem, cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    return launch_pipeline<CG>(gated_kernel<CG, OUT>, smem_set, grid, smem, stream, p, q);
}

cudaError_t launch_gated(const PersistentParams& p, const GatedTail& q, int cta_group, int dtype, int grid, size_t smem_bytes,
                         cudaStream_t stream) {
    if (cta_group == 1)
        return dtype == GEMM_BF16 ? launch_gated_typed<1, GEMM_BF16>(p, q, grid, smem_bytes, stream)
                                  : launch_gated_typed<1, GEMM_F16>(p, q, grid, smem_bytes, stream);
    return dtype == GEMM_BF16 ? launch_gated_typed<2, GEMM_BF16>(p, q, grid, smem_bytes, stream)
                              : launch_gated_typed<2, GEMM_F16>(p, q, grid, smem_bytes, stream);
}

}  // namespace dgb
