// paged_attn_host.h -- launch parameters of the paged attention kernels (internal).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "serving.h"

namespace dgb {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnSegmentCost = 2;                          // units of work a segment costs beyond its tiles
constexpr int kAttnMinUnits = 4;                             // fewest units a CTA is given while others idle

struct AttnParams {
    paged_attn_args_t a;
    int32_t heads, group, head_dim, page_size, window;
    int32_t page_shift;               // log2(page_size), or -1
    int32_t head_groups;              // segments that share a kv head: ceil(group / 8 or 16)
    int32_t segments_per_sequence;    // kv_heads * head_groups
    float score_log2;                 // |scale * k_scale| * log2(e), at least the smallest normal number
    int32_t negate;                   // scale * k_scale < 0: the queries' signs are flipped
    float* partials;                  // [CTA][2] slots: O[heads][dim], m[heads], l[heads]
    uint32_t* counters;               // [sequence][segment]: CTAs that left their partial; zero between launches
};

struct AttnVariant {
    cudaError_t (*launch)(const AttnParams&, int grid, cudaStream_t) = nullptr;
    int smem_bytes = 0, slot_floats = 0, ctas_per_sm = 0, tile_tokens = 0, heads = 0;
};

cudaError_t attn_variant_bf16(int head_dim, int group, AttnVariant* v);          // bf16 queries and cache
cudaError_t attn_variant_f16(int head_dim, int group, AttnVariant* v);           // f16 queries and cache
cudaError_t attn_variant_bf16_e4m3(int head_dim, int group, AttnVariant* v);     // bf16 queries, E4M3 cache
cudaError_t attn_variant_f16_e4m3(int head_dim, int group, AttnVariant* v);      // f16 queries, E4M3 cache

}  // namespace dgb
