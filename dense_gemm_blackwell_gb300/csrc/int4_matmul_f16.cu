// int4_matmul_f16.cu -- int4_matmul.cuh for f16 tokens.
#include "int4_matmul.cuh"

namespace dgb {

cudaError_t launch_int4_f16(const Int4Params& p, bool gated, cudaStream_t stream) { return launch_int4<__half>(p, gated, stream); }

}  // namespace dgb
