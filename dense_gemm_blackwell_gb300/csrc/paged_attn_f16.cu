// paged_attn_f16.cu -- instantiations of the paged attention kernel (paged_attn.cuh).
#include "paged_attn.cuh"

namespace dgb {

cudaError_t attn_variant_f16(int head_dim, int group, AttnVariant* v) { return attn_variant<__half, __half, false>(head_dim, group, v); }

}  // namespace dgb
