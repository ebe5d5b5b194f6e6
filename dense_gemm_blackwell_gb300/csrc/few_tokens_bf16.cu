// few_tokens_bf16.cu -- few_tokens.cuh for bf16 tokens.
#include "few_tokens.cuh"

namespace dgb {

cudaError_t launch_few_bf16(const FewParams& p, int vec, bool gated, cudaStream_t stream) {
    return launch_few<__nv_bfloat16>(p, vec, gated, stream);
}

}  // namespace dgb
