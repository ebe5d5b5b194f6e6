// int4_matmul.cu -- products of a few tokens with 4-bit weights: the entry point
// (include/feedforward.h) and how a call is laid on the device.  The kernel:
// int4_matmul.cuh.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "feedforward.h"
#include "int4_matmul.h"
#include "serving_host.h"

namespace dgb {

// The device's answer, asked for until there is one; a query that fails leaves nothing behind.
static cudaError_t resident(int k_split_log, int per_sm, int device, int64_t* clusters) {
    static std::atomic<int> known[kMaxDevices][4][3];
    std::atomic<int>* at = device < kMaxDevices ? &known[device][k_split_log][per_sm] : nullptr;
    int n = at ? at->load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        const cudaError_t e = int4_resident(k_split_log, per_sm, &n);
        if (e != cudaSuccess) return e;
        if (at) at->store(n, std::memory_order_relaxed);
    }
    *clusters = n;
    return cudaSuccess;
}

// A tile is 16 rows of W, a stage 256 bytes of each.  The CTAs of a cluster may share K: X in each CTA's shared memory is what one of
// them needs of it.  What is chosen costs the least by a count of cycles that was fitted to 560 times of 85 sizes (1, 8 and 16
// tokens, 608 to 77824 rows, K from 512 to 28672; in the mean the choice takes 1.2 % more than the best one):
// a stage takes a warp 4700 cycles where it shares the memory with all the others, 2900 where fewer than half of the device's warps
// have one, a quarter more with groups of 64, 1.9 times with groups of 32, 7 % more with 16 tokens, and longer when the shared memory
// leaves the L1 cache less room than the loads on their way take; X comes in at 13 bytes a cycle (of two CTAs an SM at less); a
// tile's sums cost 38 cycles a token, more than twice that in a cluster, a doubling of the cluster 840; 16 warps meet later than 8.
// Measured, 8 tokens x 4096 -> 4864 and 77824: two CTAs of 8 warps 8.5 and 37.7 us, in clusters of two 7.3 and 45.7, one CTA of 16
// warps 7.6 and 37.1; 16 tokens -> 77824 in clusters of two 82, one CTA 51.
gemm_status_t shape_int4(Int4Params* p, bool gated, const DeviceFacts& dev) {
    constexpr int64_t kStageK = 2 * kInt4RowBytes;
    const int64_t tiles = ((int64_t)p->n + (gated ? 7 : 15)) / (gated ? 8 : 16), stages = (p->k + kStageK - 1) / kStageK;
    const int64_t tokens = p->tokens > 8 ? 16 : 8, slot = tokens * 17 * 4;
    const int64_t chunks = p->group % 128 == 0 ? 4 : p->group % 64 == 0 ? 8 : 16;       // of a stage
    const double stage_cost = (chunks == 4 ? 1.0 : chunks == 8 ? 1.25 : 1.9) * (tokens > 8 ? 1.07 : 1.0);
    double best = 0;
    // two CTAs of 8 warps an SM, one of 16 or, of X too long for its other places, one of 8
    for (int choice = 0; choice < (best > 0 ? 2 : 3); ++choice) {
        const int per_sm = choice == 0 ? 2 : 1;
        const int64_t room = kInt4Room / per_sm, warps = choice == 1 ? 16 : 8;
        for (int ks = 0; ks <= 3 && (1 << ks) <= stages; ++ks) {
            const int64_t mine = (stages + (1 << ks) - 1) >> ks;
            const int64_t base = warps * chunks * 16 * 8 + mine * (kStageK * tokens * 2 + chunks * tokens * 4);
            int64_t at_once = per_sm * dev.sms;
            if (ks > 0) {
                const cudaError_t e = resident(ks, per_sm, dev.device, &at_once);
                if (e != cudaSuccess) return status_of(e);
                if (at_once < 1) continue;
            }
            const int64_t clusters = std::min(tiles, at_once);
            const int64_t all = (tiles + clusters - 1) / clusters;      // tiles of a cluster
            int64_t slots = 2 * warps, round_tiles = all;
            if (ks > 0) {
                const int64_t most = kInt4RoundTiles * 8 / tokens;
                slots = warps - 1 + all;
                if (all > most || base + slots * slot > room) {
                    const int64_t fit = std::min(((room - base) / slot) / 2 - (warps - 1), most / 2);
                    if (fit < 1) continue;
                    const int64_t rounds = (all + fit - 1) / fit;
                    round_tiles = (all + rounds - 1) / rounds;
                    slots = 2 * (warps - 1 + round_tiles);
                }
            }
            const int64_t smem = base + slots * slot, units = all * mine, beside = (clusters << ks) > dev.sms ? 2 : 1;
            if (smem > room) continue;
            const double cache = std::max(8.0, 256.0 - beside * (double)(smem + 1536) / 1024), full = units * (clusters << ks) > 8 * dev.sms;
            const double cost = (double)((units + warps - 1) / warps) * stage_cost * (full ? 4700 : 2900) * (1 + 0.44 * std::max(0.0, 64 / cache - 0.89)) +
                                (double)(mine * kStageK * 2 * p->tokens) / 13 * (beside > 1 ? 2.2 : 1) + 38.0 * all * p->tokens * (ks > 0 ? 2.2 : 1) +
                                840 * ks + (choice == 1 ? 1000 : 0);
            if (best > 0 && cost >= best) continue;
            best = cost;
            p->k_split_log = ks;
            p->grid = (int)(clusters << ks);
            p->round_tiles = (int)round_tiles;
            p->slots = (int)slots;
            p->warps_log = warps == 8 ? 3 : 4;
            p->smem = (int)smem;
        }
    }
    p->tokens_log = 0;
    while ((1 << p->tokens_log) < p->tokens) ++p->tokens_log;
    return best > 0 ? GEMM_OK : GEMM_ERR_UNSUPPORTED;       // X does not fit
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
    gemm_status_t s = device_facts(&dev);
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
    if ((s = shape_int4(&f, gated, dev)) != GEMM_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(a.dtype == GEMM_BF16 ? launch_int4_bf16(f, gated, st) : launch_int4_f16(f, gated, st));
}

}  // extern "C"
