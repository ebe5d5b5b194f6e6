// int4_matmul_bf16.cu -- int4_matmul.cuh for bf16 tokens.
#include "int4_matmul.cuh"

namespace dgb {

cudaError_t int4_resident(int k_split_log, int per_sm, int* clusters) { return resident_int4<__nv_bfloat16>(k_split_log, per_sm, clusters); }
cudaError_t launch_int4_bf16(const Int4Params& p, bool gated, cudaStream_t stream) { return launch_int4<__nv_bfloat16>(p, gated, stream); }

}  // namespace dgb
