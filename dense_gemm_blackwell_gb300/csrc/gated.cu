// gated.cu -- a gated pair of projections (include/feedforward.h): plans and the
// pass over the kept sums that begins the backward pass.
//
// Forward, up to 128 tokens: one wave of CTAs over W, columns dealt out evenly
// (gated_few.cu).  More: the persistent pipeline on W's 2 x features rows
// (kernels_gated.cu).  Backward: d_gate_up = [dH U act'(G), dH act(G)] in one pass
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
#include "gated_few.h"
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

// Both gradients are rounded to 16 bits once, because the products after it take 16-bit operands: at 4096 x 4096 -> 2 x 8192 bf16
// the errors of dX and dW against 64 bits are 0.0023 of their size, 0.0017 with gradients in 32 bits, which is the outputs' own
// rounding.  A second 16-bit term would double both products, 590 of the pass's 640 us.
//
// Bound by memory: 10 bytes an element of H, 4096 x 8192 in 48 us, 7.0 TB/s (the gradients are partly still in L2 when it ends).
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

}  // namespace dgb

using namespace dgb;

struct gated_plan_s {
    gated_desc_t desc;              // resolved
    gated_plan_info_t info;
    int device = 0, sms = 0;
    gemm_plan_t forward = nullptr, dx = nullptr, dw = nullptr;
    PersistentParams params;        // of the pointers below
    GatedTail tail;
    GatedFewParams tiles{};         // few tiles: what does not change from run to run, and the maps of the pointers below
    dim3 tiles_grid;
    size_t tiles_smem = 0;
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

// The kernel for few tokens takes up to 96, and up to 128 where the pipeline's tiles would cover less than half of the SMs: with more,
// its sums on their way to the stores cost what its even wave gains (4096 x 2 x 12288: 1 token 31.4 us here, 52 there, 96 37.1 and 37.9,
// 128 39.6 and 38.0; 4096 x 2 x 4096, 128 tokens: 17.4 and 23.8).  Columns and K are dealt out over one wave of clusters as costs the
// least: an SM takes in about 50 bytes a cycle and 200 cycles a K block beside; a join costs a start and what its sums cost.  (One
// wave: a 37th cluster of four CTAs, where the device held 36, doubled the time.)  Says in info.few_tiles whether it is taken.
gemm_status_t plan_few_tiles(const gated_desc_t& d, const DeviceFacts& dev, gated_plan_s* p) {
    if (d.tokens > 128 || (d.tokens > 96 && 2 * d.features >= 128 * (int64_t)dev.sms)) return GEMM_OK;
    const int64_t k_blocks = (d.k + 63) / 64, box_m = (d.tokens + 7) / 8 * 8;
    GatedFewParams& q = p->tiles;
    double best = 0;
    for (int64_t ks = 1; ks <= kGatedFewMaxSplit && ks <= k_blocks; ks *= 2) {
        int wave = 0;
        const cudaError_t e = gated_few_max_clusters(d.dtype, (int)ks, dev, &wave);
        if (e != cudaSuccess) return status_of(e);
        for (int64_t half = 8; half <= 128; half += 8) {
            if ((d.features + half - 1) / half > wave) continue;
            const double sums = (double)(box_m * 2 * half);
            const double cost = (double)((k_blocks + ks - 1) / ks) * ((box_m + 2 * half) * 128 / 50 + 200) + 0.1 * sums +
                                (ks > 1 ? 1000 + 0.1 * ks * sums : 0);
            if (best > 0 && cost >= best) continue;
            best = cost;
            q.half = (int32_t)half;
            q.k_split = (int32_t)ks;
        }
    }
    if (best == 0) return GEMM_OK;
    p->info.few_tiles = 1;
    q.M = (int32_t)d.tokens;
    q.features = (int32_t)d.features;
    q.k_blocks = (int32_t)k_blocks;
    q.box_m = (int32_t)box_m;
    q.tmem_cols = 32;
    while (q.tmem_cols < 2 * q.half) q.tmem_cols *= 2;
    q.sum_pitch = 2 * q.half + 4;
    q.ldy = d.ldh;
    q.ld_gate_up = d.ld_gate_up;
    q.act = d.activation;
    q.timeout_ns = d.wait_timeout_ns ? d.wait_timeout_ns : 2000000000ull;
    q.idesc = make_idesc(d.dtype == GEMM_BF16 ? 1u : 0u, 128u, 2u * q.half);
    // the last stage's matrix instruction reads 128 rows from its X box on: 16 KB behind the ring
    const int64_t stage = (box_m + 2 * q.half) * 128, slack = 128 * 128 + 1024, most = dev.smem_optin - 2048 - slack;
    q.stages = (int32_t)std::max<int64_t>(2, std::min<int64_t>({most / stage, (int64_t)kGatedFewMaxStages, (k_blocks + q.k_split - 1) / q.k_split}));
    // the sums lie over the ring
    const int64_t bytes = std::max(q.stages * stage, d.tokens * q.sum_pitch * 4);
    p->tiles_grid = dim3((unsigned)((d.features + q.half - 1) / q.half * q.k_split));
    p->tiles_smem = (size_t)(bytes + slack);
    return GEMM_OK;
}

// Tensor maps and pointers of a run, kept while the pointers stay the same.
gemm_status_t few_tiles_params(gated_plan_s* plan, const void* x, const void* w, void* h, void* gate_up) {
    const gated_desc_t& d = plan->desc;
    GatedFewParams& q = plan->tiles;
    gemm_status_t s = encode_rows_map(&q.tmap_x, d.dtype, x, d.k, d.tokens, d.ldx, q.box_m);
    if (s == GEMM_OK) s = encode_rows_map(&q.tmap_w, d.dtype, w, d.k, 2 * d.features, d.ldw, q.half);
    q.y = h;
    q.gate = gate_up;
    q.up = gate_up ? static_cast<uint16_t*>(gate_up) + d.features : nullptr;
    q.status = device_record(plan->forward);
    return s;
}

gemm_status_t pipeline_params(gated_plan_s* plan, const void* x, const void* w, void* h, void* gate_up) {
    const gated_desc_t& d = plan->desc;
    PersistentParams& p = plan->params;
    GatedTail& q = plan->tail;
    std::memset(&q, 0, sizeof(q));
    gemm_status_t s = product_params(plan->forward, x, w, h, &p);
    // W's rows of one kind; the output's columns
    if (s == GEMM_OK) s = encode_rows_map(&p.tmap_b, d.dtype, w, d.k, 2 * d.features, d.ldw, std::min(p.tile_n, 256) / 2);
    if (s == GEMM_OK) s = encode_rows_map(&p.tmap_d, d.dtype, h, d.features, d.tokens, d.ldh, 32);
    if (s == GEMM_OK && gate_up) s = encode_rows_map(&q.tmap_gate, d.dtype, gate_up, d.features, d.tokens, d.ld_gate_up, 32);
    if (s == GEMM_OK && gate_up)
        s = encode_rows_map(&q.tmap_up, d.dtype, static_cast<uint16_t*>(gate_up) + d.features, d.features, d.tokens, d.ld_gate_up, 32);
    q.features = (int32_t)d.features;
    q.act = d.activation;
    q.keep = gate_up != nullptr;
    return s;
}

// The pipeline's tiles where 512-wide ones of SM pairs, which the planner takes for a product of this size, would fill two waves at
// most: an epilogue that ends in half as many columns hides less behind the next tile, and whole waves count for more than tiles.  A
// wave takes so many microseconds along a K of 4096, and a launch some beside.  Fitted to 65 sizes (130 to 3000 tokens, K 1024 to
// 4096): 130 x 4096 -> 2 x 4096 19.2 us in pairs, 21.2 in single CTAs; 512 x 4096 -> 2 x 12288 68.7 us 256 wide in three waves, 78.1
// 512 wide in two; 640 x 1024 -> 2 x 3584 11.3 us in single CTAs, 15.5 in pairs.  Splitting the last wave along K, whose partial sums
// are of both kinds, cost 3 to 5 us there.  Tiles for half of the device or less share K where that saves more than the 14 us that
// the parts' join takes of a long one: 130 x 16384 -> 2 x 1024 27.6 us, 43.0 unsplit, 130 x 28672 -> 2 x 512 33.6 and 72.0; 130 x
// 6144 -> 2 x 1024, which would save 13 of its tiles' time, 19.9 and 19.0.
void choose_tiles(const gated_desc_t& d, int sms, gemm_desc_t* f) {
    const auto tiles = [&](int group, int64_t n) { return (d.tokens + 128 * group - 1) / (128 * group) * ((2 * d.features + n - 1) / n); };
    const auto waves = [&](int group, int64_t n) {
        const int64_t at_once = sms / group;
        return (double)((tiles(group, n) + at_once - 1) / at_once);
    };
    if (d.tokens <= 128 || d.features < 128 || waves(2, 512) > 2) return;
    struct Tiles { int32_t n; int group; double wave, beside; };
    double best = 0;
    for (const Tiles& o : {Tiles{512, 2, 36.5, 6.4}, Tiles{256, 2, 19.0, 6.4}, Tiles{128, 2, 11.2, 6.4}, Tiles{256, 1, 23.5, 5.0}, Tiles{128, 1, 15.0, 5.0}}) {
        const double cost = waves(o.group, o.n) * o.wave * (double)d.k / 4096 + o.beside;
        if (best > 0 && cost >= best) continue;
        best = cost;
        const int64_t parts = sms / o.group / tiles(o.group, o.n);
        const bool split = o.n == 512 || (parts > 1 && o.wave * (double)d.k / 4096 * (1.0 - 1.0 / (double)parts) > 14);
        f->tile_n = o.n;
        f->flags = GEMM_FLAG_NO_SINGLE_CTA | (o.group == 2 ? GEMM_FLAG_CTA_GROUP_2 : GEMM_FLAG_CTA_GROUP_1) | (split ? 0u : GEMM_FLAG_NO_STREAM_K);
    }
}

// The gradients' products have MN-major operands, for which the planner does not choose 512-wide tiles by itself. They take them where
// those fill their last wave well enough to make up for its not being split along K as that of 256-wide tiles is: 16384 x 4096 x 4096
// (7 waves, 96 % full) 298 us, 352 with 256; the whole backward pass of 2048 and 8192 tokens, 4096 -> 2 x 8192, 323 and 1247 us, 349 and
// 1356 with 256 (in a graph; a loop of calls under the power cap takes a tenth more). Along a short K the unsplit last wave costs more: at 84 % 4096 x 4096 x 16384 still gains (628 us for the whole pass at
// 4096 tokens, 642 with 256 in that product), 16384 x 2048 x 2048 loses (205 us, 187 with 256).  Up to 128 rows are lone CTAs' tiles,
// for which waves of pairs say nothing: 64 x 32768 x 16384 153 us in the planner's tiles, 189 with 512, 64 x 36864 x 2048 28 and 43.
int32_t mn_tile(const gemm_desc_t& g, int sms) {
    if (g.M <= 128) return 0;
    const int64_t tiles = (g.M + 255) / 256 * ((g.N + 511) / 512), pairs = sms / 2, waves = (tiles + pairs - 1) / pairs;
    return g.K >= 1024 && g.N % 512 == 0 && 10 * tiles >= (g.K >= 4096 ? 8 : 9) * waves * pairs ? 512 : 0;
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
    gemm_desc_t f = g;
    f.M = d.tokens;
    f.N = 2 * d.features;
    f.K = d.k;
    f.dtype_d = d.dtype;
    f.lda = d.ldx;
    f.ldb = d.ldw;
    if (d.tokens > 0 && !forced && (s = plan_few_tiles(d, dev, p)) != GEMM_OK) {
        gated_plan_destroy(p);
        return s;
    }
    f.flags = d.flags | GEMM_FLAG_NO_SINGLE_CTA;
    if (p->info.few_tiles) f.flags |= GEMM_FLAG_NO_STREAM_K;       // the product's plan holds the error record only
    f.tile_n = d.tile_n == 0 && d.features < 128 ? 128 : d.tile_n;     // tiles hold whole 64-column chunks of both kinds
    f.stages = d.stages;
    f.max_ctas = d.max_ctas;
    if (!forced && !p->info.few_tiles) choose_tiles(d, dev.sms, &f);
    s = make_product(&p->forward, &p->info.product, f);
    if (s == GEMM_OK && p->info.few_tiles) {
        // what runs instead
        gemm_plan_info_t& info = p->info.product;
        const GatedFewParams& q = p->tiles;
        info.cta_group = 1;
        info.tile_m = 128;
        info.tile_n = 2 * q.half;
        info.tile_k = 64;
        info.stages = q.stages;
        info.tmem_stages = 1;
        info.tmem_cols = q.tmem_cols;
        info.grid = (int32_t)p->tiles_grid.x;
        info.block_threads = 192;
        info.num_tiles = p->tiles_grid.x / q.k_split;
        info.stage_bytes = (q.box_m + 2 * q.half) * 128;
        info.pipeline_bytes = info.stages * info.stage_bytes + 8 * (2 * info.stages + 1) + 4;
        info.smem_bytes = (int64_t)p->tiles_smem;
        info.epilogue = 1;
        p->info.k_split = q.k_split;
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
        x.tile_n = mn_tile(x, dev.sms);
        w.tile_n = mn_tile(w, dev.sms);
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
    const void* now[4] = {x, w, h, gate_up};
    if (!plan->params_valid || std::memcmp(now, plan->ptrs, sizeof(now)) != 0) {
        plan->params_valid = false;
        s = plan->info.few_tiles ? few_tiles_params(plan, x, w, h, gate_up) : pipeline_params(plan, x, w, h, gate_up);
        if (s != GEMM_OK) return s;
        std::memcpy(plan->ptrs, now, sizeof(now));
        plan->params_valid = true;
    }
    if (plan->info.few_tiles) return status_of(launch_gated_few(plan->tiles, d.dtype, plan->tiles_grid, plan->tiles_smem, st));
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

}  // extern "C"
