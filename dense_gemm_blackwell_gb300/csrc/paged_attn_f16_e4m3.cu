// paged_attn_f16_e4m3.cu -- instantiations of the paged attention kernel (paged_attn.cuh).
#include "paged_attn.cuh"

namespace dgb {

cudaError_t attn_variant_f16_e4m3(int head_dim, int group, AttnVariant* v) { return attn_variant<__half, __half, true>(head_dim, group, v); }

}  // namespace dgb
