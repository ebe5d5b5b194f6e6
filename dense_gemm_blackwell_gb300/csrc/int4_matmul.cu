// int4_matmul.cu -- products of a few tokens with 4-bit weights: the entry point
// (include/feedforward.h) and how a call is laid on the device.  The kernel:
// int4_matmul.cuh.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "feedforward.h"
#include "int4_matmul.h"
#include "serving_host.h"

namespace dgb {

// A tile is 16 rows of W, a stage 256 bytes of each.  Clusters may share K, warps of a block a tile; what is chosen costs the least
// by a rough count of cycles: a stage takes a warp 1600 with one block on the SM and 2500 with two (twice that with groups of 32,
// whose factors change every 32 elements; a third more with 16 tokens), a tile's end 600 and 800 more for every doubling of a
// cluster; X comes into a block's shared memory at 24 bytes a cycle, and the shared memory it takes is missed as L1 cache.
bool shape_int4(Int4Params* p, bool gated, int sms) {
    constexpr int64_t kStageK = 2 * kInt4RowBytes;
    const int64_t tiles = ((int64_t)p->n + (gated ? 7 : 15)) / (gated ? 8 : 16), stages = (p->k + kStageK - 1) / kStageK;
    const int64_t tokens = p->tokens > 8 ? 16 : 8, sums = 2 * kInt4Warps * tokens * 17 * 4;
    const int64_t chunks = p->group % 128 == 0 ? 4 : p->group % 64 == 0 ? 8 : 16;       // of a stage
    const int64_t factors = kInt4Warps * chunks * 16 * 8;
    const double stage_cost = (chunks == 4 ? 1.0 : chunks == 8 ? 1.3 : 2.0) * (tokens > 8 ? 1.35 : 1.0);
    double best = 0;
    // two blocks an SM, or, of X too long for that, one
    for (int per_sm = 2; per_sm >= 1 && best == 0; --per_sm) {
        for (int ks = 0; ks <= 3 && (1 << ks) <= stages; ++ks) {
            const int64_t clusters = (per_sm * sms) >> ks, mine = (stages + (1 << ks) - 1) >> ks;
            const int64_t smem = sums + factors + mine * (kStageK * tokens * 2 + chunks * tokens * 4);
            if (smem > (per_sm == 2 ? 112 : 224) * 1024) continue;
            for (int kw = 0; (1 << kw) <= kInt4Warps; ++kw) {
                const int64_t per_round = kInt4Warps >> kw, blocks = std::min((tiles + per_round - 1) / per_round, clusters);
                const int64_t rounds = (tiles + per_round * blocks - 1) / (per_round * blocks), per_tile = (mine + (1 << kw) - 1) >> kw;
                const double beside = (blocks << ks) > sms ? 1.0 : 0.5;        // how full an SM is
                const double cost = (double)rounds * (per_tile * stage_cost * (700 + 1800 * beside) + 600 + 800 * ks) +
                                    (double)(mine * kStageK * 2) * (p->tokens / 24.0 + tokens / 60.0);
                if (best > 0 && cost >= best) continue;
                best = cost;
                p->k_split_log = ks;
                p->k_warps_log = kw;
                p->rounds = (int)rounds;
                p->grid = (int)(blocks << ks);
                p->smem = (int)smem;
            }
        }
    }
    p->tokens_log = 0;
    while ((1 << p->tokens_log) < p->tokens) ++p->tokens_log;
    return best > 0;
}

static bool type16(int32_t t) { return t == GEMM_BF16 || t == GEMM_F16; }

// A leading dim: 0 = packed; false where rows would overlap.
static bool settle(int64_t& ld, int64_t least) {
    if (ld == 0) ld = least;
    return ld >= least;
}

}  // namespace dgb

using namespace dgb;

extern "C" {

gemm_status_t int4_matmul_run(const int4_matmul_args_t* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_INVALID_ARG;
    int4_matmul_args_t a = *args;
    if (a.tokens < 0 || a.n < 1 || a.k < 1 || a.group < 1) return GEMM_ERR_INVALID_ARG;
    if (a.activation < GATED_SILU || a.activation > GATED_NONE) return GEMM_ERR_INVALID_ARG;
    const bool gated = a.activation != GATED_NONE;
    if (!type16(a.dtype) || a.tokens > kInt4TokensMax || a.k % 2 != 0 || a.group % 32 != 0 || a.n > kInt4RowsMax)
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
    Int4Params f{};
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
    if (!shape_int4(&f, gated, dev.sms)) return GEMM_ERR_UNSUPPORTED;       // X does not fit
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(a.dtype == GEMM_BF16 ? launch_int4_bf16(f, gated, st) : launch_int4_f16(f, gated, st));
}

}  // extern "C"
