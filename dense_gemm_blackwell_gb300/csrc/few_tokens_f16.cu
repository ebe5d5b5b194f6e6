// few_tokens_f16.cu -- few_tokens.cuh for f16 tokens.
#include "few_tokens.cuh"

namespace dgb {

cudaError_t launch_few_f16(const FewParams& p, int vec, bool gated, cudaStream_t stream) {
    return launch_few<__half>(p, vec, gated, stream);
}

}  // namespace dgb
