// gated.cu -- a gated pair of projections (include/feedforward.h): plans, the
// pass over the kept sums that begins the backward pass, and the 4-bit products'
// entry point, which shares the streaming kernel.
//
// Forward, more than kFewTokensMax tokens: the persistent pipeline on W's 2 x
// features rows (kernels_gated.cu).  Up to that many: one stream over W
// (few_tokens.cuh).  Backward: d_gate_up = [dH U act'(G), dH act(G)] in one pass
// over memory, then two of the library's products, d_gate_up W (W as an N-major
// operand, K = 2 features) and d_gate_up^T X (both operands M- and N-major).
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>

#include <cuda_runtime.h>

#include "activation.cuh"
#include "common.cuh"
#include "elem.cuh"
#include "feedforward.h"
#include "few_tokens.h"
#include "launch.h"
#include "serving_host.h"

namespace dgb {

constexpr int kSlopeThreads = 256;

struct SlopeParams {
    const uint16_t* dh;
    const uint16_t* gate_up;
    uint16_t* d_gate_up;
    int64_t ldh, ld_gate_up;
    int64_t vectors;            // tokens x features / 8
    int32_t features, act;
};

// Bound by memory: 10 bytes an element of H.
template <typename T>
__global__ void __launch_bounds__(kSlopeThreads) gated_slope_kernel(const __grid_constant__ SlopeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = p.features / 8;
    for (int64_t i = (int64_t)blockIdx.x * kSlopeThreads + threadIdx.x; i < p.vectors; i += (int64_t)gridDim.x * kSlopeThreads) {
        const int64_t row = i / per_row;
        const int64_t col = (i - row * per_row) * 8;
        const int64_t at = row * p.ld_gate_up + col;
        float d[8], g[8], u[8], dg[8], du[8];
        unpack8<T>(__ldcs(reinterpret_cast<const uint4*>(p.dh + row * p.ldh + col)), d);
        unpack8<T>(__ldcs(reinterpret_cast<const uint4*>(p.gate_up + at)), g);
        unpack8<T>(__ldcs(reinterpret_cast<const uint4*>(p.gate_up + at + p.features)), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 a = activate_with_slope(p.act, g[j]);
            dg[j] = d[j] * u[j] * a.y;
            du[j] = d[j] * a.x;
        }
        *reinterpret_cast<uint4*>(p.d_gate_up + at) = round8<T>(dg);
        *reinterpret_cast<uint4*>(p.d_gate_up + at + p.features) = round8<T>(du);
    }
}

// A tile is 16 rows of W, a stage 256 bytes of each.  Clusters share K as often as X (in whole stages, 8 or 16 tokens) needs for two
// blocks to fit an SM, and further while that leaves no more blocks than fit the device and every warp a stage.  Then as many warps
// share a tile as leaves a block the fewest stages in sequence, a tile's end counted as half a stage.
bool shape_few(FewParams* p, bool gated, bool four_bits, int sms) {
    constexpr int64_t kSmemMax = 112 * 1024;
    const int64_t tiles = ((int64_t)p->n + (gated ? 7 : 15)) / (gated ? 8 : 16);
    const int64_t stage_k = four_bits ? 2 * kFewRowBytes : kFewRowBytes / 2, stages = (p->k + stage_k - 1) / stage_k;
    const int64_t tokens = p->tokens > 8 ? 16 : 8, sums = 2 * kFewWarps * tokens * 17 * 4;
    auto x_bytes = [&](int64_t ks) { return (stages + ks - 1) / ks * stage_k * tokens * 2; };
    int ks = 0;
    while (ks <= 3 && sums + x_bytes(1 << ks) > kSmemMax) ++ks;
    if (ks > 3) return false;
    while (ks < 3 && (tiles << (ks + 1)) <= 2 * sms && stages >= (2 * kFewWarps) << ks) ++ks;
    const int64_t clusters = (2 * sms) >> ks, mine = (stages + (1 << ks) - 1) >> ks;
    int64_t best = INT64_MAX;
    for (int kw = 0; (1 << kw) <= kFewWarps; ++kw) {
        const int64_t at_once = clusters * (kFewWarps >> kw), rounds = (tiles + at_once - 1) / at_once;
        const int64_t cost = rounds * (2 * ((mine + (1 << kw) - 1) >> kw) + 1);
        if (cost < best) {
            best = cost;
            p->k_warps_log = kw;
        }
    }
    const int per_round = kFewWarps >> p->k_warps_log;
    const int64_t blocks = std::min<int64_t>((tiles + per_round - 1) / per_round, clusters);
    p->k_split_log = ks;
    p->rounds = (int)((tiles + per_round * blocks - 1) / (per_round * blocks));
    p->grid = (int)(blocks << ks);
    p->smem = (int)(sums + x_bytes(1 << ks));
    return true;
}

static cudaError_t launch_few(const FewParams& p, int dtype, int vec, bool gated, cudaStream_t stream) {
    return dtype == GEMM_BF16 ? launch_few_bf16(p, vec, gated, stream) : launch_few_f16(p, vec, gated, stream);
}

}  // namespace dgb

using namespace dgb;

struct gated_plan_s {
    gated_desc_t desc;              // resolved
    gated_plan_info_t info;
    int device = 0, sms = 0;
    gemm_plan_t forward = nullptr, dx = nullptr, dw = nullptr;
    PersistentParams params;        // of the pointers below
    GatedTail tail;
    FewParams few{};                // streamed: what does not change from run to run
    const void* ptrs[4] = {nullptr, nullptr, nullptr, nullptr};
    bool params_valid = false;
};

namespace {

constexpr uint32_t kGatedFlags = GEMM_FLAG_CTA_GROUP_1 | GEMM_FLAG_CTA_GROUP_2 | GEMM_FLAG_NO_STREAM_K | GEMM_FLAG_STAGE_K1 | GEMM_FLAG_STAGE_K2;

bool type16(int32_t t) { return t == GEMM_BF16 || t == GEMM_F16; }

bool settle(int64_t& ld, int64_t least) {
    if (ld == 0) ld = least;
    return ld >= least;
}

gemm_status_t resolve_gated(gated_desc_t* d) {
    if (d->tokens < 0 || d->features < 1 || d->k < 1) return GEMM_ERR_INVALID_ARG;
    if (d->activation < GATED_SILU || d->activation > GATED_GELU_TANH) return GEMM_ERR_INVALID_ARG;
    if (d->gradients != 0 && d->gradients != 1) return GEMM_ERR_INVALID_ARG;
    if (!type16(d->dtype)) return GEMM_ERR_UNSUPPORTED;
    if (d->gradients && d->dtype_dw != d->dtype && d->dtype_dw != GEMM_F32) return GEMM_ERR_UNSUPPORTED;
    if (d->features % 8 != 0 || d->tokens > INT32_MAX || d->features > INT32_MAX / 2 || d->k > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
    if (!settle(d->ldx, d->k) || !settle(d->ldw, d->k) || !settle(d->ldh, d->features) || !settle(d->ld_gate_up, 2 * d->features) ||
        !settle(d->ld_dx, d->k) || !settle(d->ld_dw, d->k))
        return GEMM_ERR_INVALID_ARG;
    if (!all_multiples(8, {d->ldx, d->ldw, d->ldh, d->ld_gate_up})) return GEMM_ERR_ALIGNMENT;
    if (d->gradients && (d->ld_dx % 8 != 0 || d->ld_dw % (d->dtype_dw == GEMM_F32 ? 4 : 8) != 0)) return GEMM_ERR_ALIGNMENT;
    if (d->flags & ~kGatedFlags) return GEMM_ERR_UNSUPPORTED;
    if (d->tile_n != 0 && d->tile_n != 128 && d->tile_n != 256 && d->tile_n != 512) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

gemm_status_t make_product(gemm_plan_t* plan, gemm_plan_info_t* info, const gemm_desc_t& g) {
    const gemm_status_t s = gemm_plan_create(plan, &g);
    return s == GEMM_OK ? gemm_plan_info(*plan, info) : s;
}

}  // namespace

extern "C" {

gemm_status_t gated_plan_create(gated_plan_t* out, const gated_desc_t* desc) {
    if (!out || !desc) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    gated_desc_t d = *desc;
    gemm_status_t s = resolve_gated(&d);
    if (s != GEMM_OK) return s;
    DeviceFacts dev;
    if ((s = device_facts(&dev)) != GEMM_OK) return s;
    gated_plan_s* p = new (std::nothrow) gated_plan_s();
    if (!p) return GEMM_ERR_RESOURCES;
    p->desc = d;
    std::memset(&p->info, 0, sizeof(p->info));
    p->device = dev.device;
    p->sms = dev.sms;
    gemm_desc_t g{};
    g.batch = 1;
    g.dtype_a = g.dtype_b = d.dtype;
    g.wait_timeout_ns = d.wait_timeout_ns;
    const bool forced = d.flags != 0 || d.tile_n != 0 || d.stages != 0 || d.max_ctas != 0;
    if (d.tokens <= kFewTokensMax && !forced) {
        p->few.tokens = (int32_t)d.tokens;
        p->few.k = (int32_t)d.k;
        p->few.n = (int32_t)d.features;
        p->info.streamed = shape_few(&p->few, true, false, dev.sms);
        if (p->info.streamed) p->info.k_split = 1 << p->few.k_split_log;
    }
    if (!p->info.streamed) {
        gemm_desc_t f = g;
        f.M = d.tokens;
        f.N = 2 * d.features;
        f.K = d.k;
        f.dtype_d = d.dtype;
        f.lda = d.ldx;
        f.ldb = d.ldw;
        f.flags = d.flags | GEMM_FLAG_NO_SINGLE_CTA;
        f.tile_n = d.tile_n == 0 && d.features < 128 ? 128 : d.tile_n;     // tiles hold whole 64-column chunks of both kinds
        f.stages = d.stages;
        f.max_ctas = d.max_ctas;
        s = make_product(&p->forward, &p->info.product, f);
    }
    if (s == GEMM_OK && d.gradients) {
        gemm_desc_t x = g;      // d_x [tokens, k] = d_gate_up [tokens, 2 features] * W, W's rows the contraction
        x.M = d.tokens;
        x.N = d.k;
        x.K = 2 * d.features;
        x.dtype_d = d.dtype;
        x.major_b = GEMM_MN_MAJOR;
        x.lda = d.ld_gate_up;
        x.ldb = d.ldw;
        x.ldd = d.ld_dx;
        gemm_desc_t w = g;      // d_w [2 features, k] = d_gate_up^T X, tokens the contraction
        w.M = 2 * d.features;
        w.N = d.k;
        w.K = d.tokens;
        w.dtype_d = d.dtype_dw;
        w.major_a = w.major_b = GEMM_MN_MAJOR;
        w.lda = d.ld_gate_up;
        w.ldb = d.ldx;
        w.ldd = d.ld_dw;
        s = make_product(&p->dx, &p->info.dx, x);
        if (s == GEMM_OK) s = make_product(&p->dw, &p->info.dw, w);
    }
    if (s != GEMM_OK) {
        gated_plan_destroy(p);
        return s;
    }
    p->info.workspace_bytes = p->info.product.workspace_bytes + p->info.dx.workspace_bytes + p->info.dw.workspace_bytes;
    *out = p;
    return GEMM_OK;
}

gemm_status_t gated_plan_info(gated_plan_t plan, gated_plan_info_t* info) {
    if (!plan || !info) return GEMM_ERR_INVALID_ARG;
    *info = plan->info;
    return GEMM_OK;
}

gemm_status_t gated_run(gated_plan_t plan, const void* x, const void* w, void* h, void* gate_up, gemm_stream_t stream) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    gemm_status_t s = check_device(plan->device);
    if (s != GEMM_OK) return s;
    const gated_desc_t& d = plan->desc;
    if (d.tokens == 0) return GEMM_OK;
    if (!x || !w || !h) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {x, w, h, gate_up})) return GEMM_ERR_ALIGNMENT;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (plan->info.streamed) {
        FewParams f = plan->few;
        f.x = x;
        f.w = w;
        f.y = h;
        f.gate = gate_up;
        f.up = gate_up ? static_cast<uint16_t*>(gate_up) + d.features : nullptr;
        f.ldx = d.ldx;
        f.ldw_bytes = 2 * d.ldw;
        f.ldy = d.ldh;
        f.ld_gate_up = d.ld_gate_up;
        f.act = d.activation;
        return status_of(launch_few(f, d.dtype, 0, true, st));
    }
    const void* now[4] = {x, w, h, gate_up};
    if (!plan->params_valid || std::memcmp(now, plan->ptrs, sizeof(now)) != 0) {
        plan->params_valid = false;
        if ((s = product_params(plan->forward, x, w, h, &plan->params)) != GEMM_OK) return s;
        PersistentParams& p = plan->params;
        GatedTail& q = plan->tail;
        std::memset(&q, 0, sizeof(q));
        // W's rows of one kind; the output's columns
        s = encode_rows_map(&p.tmap_b, d.dtype, w, d.k, 2 * d.features, d.ldw, std::min(p.tile_n, 256) / 2);
        if (s == GEMM_OK) s = encode_rows_map(&p.tmap_d, d.dtype, h, d.features, d.tokens, d.ldh, 32);
        if (s == GEMM_OK && gate_up) {
            s = encode_rows_map(&q.tmap_gate, d.dtype, gate_up, d.features, d.tokens, d.ld_gate_up, 32);
            if (s == GEMM_OK)
                s = encode_rows_map(&q.tmap_up, d.dtype, static_cast<uint16_t*>(gate_up) + d.features, d.features, d.tokens, d.ld_gate_up, 32);
        }
        if (s != GEMM_OK) return s;
        q.features = (int32_t)d.features;
        q.act = d.activation;
        q.keep = gate_up != nullptr;
        std::memcpy(plan->ptrs, now, sizeof(now));
        plan->params_valid = true;
    }
    return status_of(launch_gated(plan->params, plan->tail, plan->info.product.cta_group, d.dtype, plan->info.product.grid,
                                  (size_t)plan->info.product.smem_bytes, st));
}

gemm_status_t gated_backward(gated_plan_t plan, const gated_grads_t* args, gemm_stream_t stream) {
    if (!plan || !args || !plan->desc.gradients) return GEMM_ERR_INVALID_ARG;
    gemm_status_t s = check_device(plan->device);
    if (s != GEMM_OK) return s;
    const gated_desc_t& d = plan->desc;
    const gated_grads_t& a = *args;
    if (!all_aligned(16, {a.d_h, a.x, a.w, a.gate_up, a.d_gate_up, a.d_x, a.d_w})) return GEMM_ERR_ALIGNMENT;
    if (d.tokens > 0) {
        if (!a.d_h || !a.gate_up || !a.d_gate_up || (a.d_x && !a.w) || (a.d_w && !a.x)) return GEMM_ERR_INVALID_ARG;
        SlopeParams p{};
        p.dh = static_cast<const uint16_t*>(a.d_h);
        p.gate_up = static_cast<const uint16_t*>(a.gate_up);
        p.d_gate_up = static_cast<uint16_t*>(a.d_gate_up);
        p.ldh = d.ldh;
        p.ld_gate_up = d.ld_gate_up;
        p.vectors = d.tokens * (d.features / 8);
        p.features = (int32_t)d.features;
        p.act = d.activation;
        const dim3 blocks((unsigned)std::min<int64_t>((p.vectors + kSlopeThreads - 1) / kSlopeThreads, (int64_t)plan->sms * 8));
        cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
        const cudaError_t e = d.dtype == GEMM_BF16
                                  ? launch_dependent(gated_slope_kernel<__nv_bfloat16>, blocks, dim3(kSlopeThreads), 0, st, p)
                                  : launch_dependent(gated_slope_kernel<__half>, blocks, dim3(kSlopeThreads), 0, st, p);
        if (e != cudaSuccess) return status_of(e);
    }
    if (a.d_x && (s = gemm_run(plan->dx, a.d_gate_up, a.w, a.d_x, nullptr, nullptr, stream)) != GEMM_OK) return s;
    if (a.d_w && (s = gemm_run(plan->dw, a.d_gate_up, a.x, a.d_w, nullptr, nullptr, stream)) != GEMM_OK) return s;
    return GEMM_OK;
}

gemm_status_t gated_sync_status(gated_plan_t plan, gemm_stream_t stream, gemm_device_error_t* out) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    gemm_device_error_t first{};
    gemm_status_t worst = GEMM_OK;
    for (gemm_plan_t product : {plan->forward, plan->dx, plan->dw}) {
        if (!product) continue;
        gemm_device_error_t rec{};
        const gemm_status_t s = gemm_sync_status(product, stream, &rec);
        if (worst == GEMM_OK && s != GEMM_OK) {
            worst = s;
            first = rec;
        }
    }
    if (!plan->forward && !plan->dx) worst = status_of(cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)));
    if (out) *out = first;
    return worst;
}

gemm_status_t gated_plan_destroy(gated_plan_t plan) {
    if (!plan) return GEMM_OK;
    gemm_status_t worst = GEMM_OK;
    for (gemm_plan_t product : {plan->forward, plan->dx, plan->dw}) {
        const gemm_status_t s = gemm_plan_destroy(product);
        if (worst == GEMM_OK) worst = s;
    }
    delete plan;
    return worst;
}

gemm_status_t int4_matmul_run(const int4_matmul_args_t* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_INVALID_ARG;
    int4_matmul_args_t a = *args;
    if (a.tokens < 0 || a.n < 1 || a.k < 1 || a.group < 1) return GEMM_ERR_INVALID_ARG;
    if (a.activation < GATED_SILU || a.activation > GATED_NONE) return GEMM_ERR_INVALID_ARG;
    const bool gated = a.activation != GATED_NONE;
    if (!type16(a.dtype) || a.tokens > kFewTokensMax || a.k % 2 != 0 || a.group % 32 != 0 || (gated && a.n > INT32_MAX / 2))
        return GEMM_ERR_UNSUPPORTED;
    const int64_t groups = ((int64_t)a.k + a.group - 1) / a.group;
    if (!settle(a.ldx, a.k) || !settle(a.ld_codes, a.k / 2) || !settle(a.ld_scales, groups) || !settle(a.ld_zeros, groups) || !settle(a.ldy, a.n))
        return GEMM_ERR_INVALID_ARG;
    if (a.tokens == 0) return GEMM_OK;
    if (!a.x || !a.codes || !a.scales || !a.y) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {a.x, a.codes}) || !all_aligned(2, {a.scales, a.y}) || (a.tokens > 1 && a.ldx % 8 != 0) ||
        ((a.n > 1 || gated) && a.ld_codes % 16 != 0))
        return GEMM_ERR_ALIGNMENT;
    DeviceFacts dev;
    const gemm_status_t s = device_facts(&dev);
    if (s != GEMM_OK) return s;
    FewParams f{};
    f.x = a.x;
    f.w = a.codes;
    f.scales = a.scales;
    f.zeros = a.zeros;
    f.y = a.y;
    f.ldx = a.ldx;
    f.ldw_bytes = a.ld_codes;
    f.ld_scales = a.ld_scales;
    f.ld_zeros = a.ld_zeros;
    f.ldy = a.ldy;
    f.tokens = a.tokens;
    f.k = a.k;
    f.n = a.n;
    f.group = a.group;
    f.act = a.activation;
    f.group_magic = (uint32_t)std::min<uint64_t>(UINT32_MAX, (1ull << 32) / (uint32_t)(a.group / 32));
    if (!shape_few(&f, gated, true, dev.sms)) return GEMM_ERR_UNSUPPORTED;
    const int vec = a.group % 128 == 0 ? 4 : a.group % 64 == 0 ? 2 : 1;
    return status_of(launch_few(f, a.dtype, vec, gated, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
