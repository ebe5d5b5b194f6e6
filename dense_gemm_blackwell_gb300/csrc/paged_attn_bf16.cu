// paged_attn_bf16.cu -- instantiations of the paged attention kernel (paged_attn.cuh).
#include "paged_attn.cuh"

namespace dgb {

cudaError_t attn_variant_bf16(int head_dim, int group, AttnVariant* v) { return attn_variant<__nv_bfloat16, __nv_bfloat16, false>(head_dim, group, v); }

}  // namespace dgb
