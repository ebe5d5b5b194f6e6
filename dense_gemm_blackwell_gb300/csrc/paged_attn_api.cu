// paged_attn_api.cu -- host side of the paged attention operator (include/serving.h): plans, checks and launches.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <new>

#include "paged_attn_host.h"
#include "serving.h"
#include "serving_host.h"

using namespace dgb;

struct paged_attn_plan_s {
    paged_attn_desc_t desc;
    paged_attn_plan_info_t info;
    AttnVariant variant;
    int device;
    int32_t group, head_groups, page_shift;
    void* memory;             // counters, then partials
    int64_t counter_bytes;
};

namespace {

gemm_status_t check_desc(const paged_attn_desc_t& d) {
    if (d.max_batch < 0 || d.heads < 1 || d.kv_heads < 1 || d.head_dim < 1 || d.page_size < 1 || d.window < 0 || d.max_ctas < 0)
        return GEMM_ERR_INVALID_ARG;
    if (d.heads % d.kv_heads != 0) return GEMM_ERR_INVALID_ARG;
    if (d.dtype != GEMM_BF16 && d.dtype != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    if (d.dtype_cache != d.dtype && d.dtype_cache != GEMM_E4M3) return GEMM_ERR_UNSUPPORTED;
    if (d.head_dim > 256 || d.head_dim % (d.dtype_cache == GEMM_E4M3 ? 16 : 8) != 0) return GEMM_ERR_UNSUPPORTED;
    if (d.heads > (1 << 16) || d.max_batch > (1 << 20)) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t paged_attn_plan_create(paged_attn_plan_t* out, const paged_attn_desc_t* desc) {
    if (!out || !desc) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    gemm_status_t s = check_desc(*desc);
    if (s != GEMM_OK) return s;
    DeviceFacts dev;
    if ((s = device_facts(&dev)) != GEMM_OK) return s;
    AttnVariant v;
    const int group = desc->heads / desc->kv_heads;
    const bool fp8 = desc->dtype_cache == GEMM_E4M3;
    cudaError_t e = desc->dtype == GEMM_BF16
                        ? (fp8 ? attn_variant_bf16_e4m3(desc->head_dim, group, &v) : attn_variant_bf16(desc->head_dim, group, &v))
                        : (fp8 ? attn_variant_f16_e4m3(desc->head_dim, group, &v) : attn_variant_f16(desc->head_dim, group, &v));
    if (e != cudaSuccess) return status_of(e);
    if (v.ctas_per_sm < 1) return GEMM_ERR_RESOURCES;
    paged_attn_plan_s* p = new (std::nothrow) paged_attn_plan_s();
    if (!p) return GEMM_ERR_RESOURCES;
    p->desc = *desc;
    p->variant = v;
    p->device = dev.device;
    p->group = group;
    p->head_groups = (group + v.heads - 1) / v.heads;
    p->page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (desc->page_size == (1 << i)) p->page_shift = i;
    int grid = dev.sms * v.ctas_per_sm;
    if (desc->max_ctas > 0 && desc->max_ctas < grid) grid = desc->max_ctas;
    p->counter_bytes = ((int64_t)desc->max_batch * desc->kv_heads * p->head_groups * 4 + 255) / 256 * 256;
    const int64_t partial_bytes = (int64_t)grid * 2 * v.slot_floats * 4;
    p->info.grid = grid;
    p->info.tile_tokens = v.tile_tokens;
    p->info.head_groups = p->head_groups;
    p->info.smem_bytes = v.smem_bytes;
    p->info.workspace_bytes = p->counter_bytes + partial_bytes;
    if ((e = cudaMalloc(&p->memory, (size_t)p->info.workspace_bytes)) != cudaSuccess) {
        delete p;
        return status_of(e);
    }
    if ((e = clear_now(p->memory, (size_t)p->counter_bytes)) != cudaSuccess) {
        cudaFree(p->memory);
        delete p;
        return status_of(e);
    }
    *out = p;
    return GEMM_OK;
}

gemm_status_t paged_attn_plan_info(paged_attn_plan_t plan, paged_attn_plan_info_t* info) {
    if (!plan || !info) return GEMM_ERR_INVALID_ARG;
    *info = plan->info;
    return GEMM_OK;
}

gemm_status_t paged_attn_run(paged_attn_plan_t plan, const paged_attn_args_t* args, gemm_stream_t stream) {
    if (!plan || !args) return GEMM_ERR_INVALID_ARG;
    const paged_attn_desc_t& d = plan->desc;
    const paged_attn_args_t& a = *args;
    if (a.batch < 0 || a.batch > d.max_batch || a.table_width < 0 || a.num_pages < 0) return GEMM_ERR_INVALID_ARG;
    if (a.batch == 0) return GEMM_OK;
    const gemm_status_t here = check_device(plan->device);
    if (here != GEMM_OK) return here;
    if (!a.q || !a.out || !a.lengths) return GEMM_ERR_INVALID_ARG;
    if (a.table_width > 0 && (!a.block_table || !a.k_cache || !a.v_cache || a.table_stride < 0)) return GEMM_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale) || !std::isfinite(a.k_scale) || !std::isfinite(a.v_scale)) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {a.q, a.out, a.k_cache, a.v_cache})) return GEMM_ERR_ALIGNMENT;
    if (!all_multiples(8, {a.q_batch, a.q_head, a.out_batch, a.out_head})) return GEMM_ERR_ALIGNMENT;
    // cache rows are copied in 16-byte pieces
    const int piece = d.dtype_cache == GEMM_E4M3 ? 16 : 8;
    if (!all_multiples(piece, {a.k_page, a.k_place, a.k_head, a.v_page, a.v_place, a.v_head})) return GEMM_ERR_ALIGNMENT;
    AttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.a = a;
    p.heads = d.heads;
    p.group = plan->group;
    p.head_dim = d.head_dim;
    p.page_size = d.page_size;
    p.page_shift = plan->page_shift;
    p.window = d.window;
    p.head_groups = plan->head_groups;
    p.segments_per_sequence = d.kv_heads * plan->head_groups;
    const double scale = (double)a.scale * (double)a.k_scale;
    p.negate = scale < 0;
    // a scale of zero becomes the smallest normal number, so that masked scores (-inf) times it stay -inf
    p.score_log2 = std::max((float)(std::fabs(scale) * 1.4426950408889634), FLT_MIN);
    p.counters = static_cast<uint32_t*>(plan->memory);
    p.partials = reinterpret_cast<float*>(static_cast<char*>(plan->memory) + plan->counter_bytes);
    return status_of(plan->variant.launch(p, plan->info.grid, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t paged_attn_plan_destroy(paged_attn_plan_t plan) {
    if (!plan) return GEMM_OK;
    const cudaError_t e = cudaFree(plan->memory);
    delete plan;
    return status_of(e);
}

}  // extern "C"
