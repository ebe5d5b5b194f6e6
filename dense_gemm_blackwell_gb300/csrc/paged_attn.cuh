// paged_attn.cuh -- attention of one new token per sequence over a paged
// key-value cache (include/serving.h): kernel and launcher, one translation
// unit per pair of query and cache types (paged_attn_bf16.cu, paged_attn_f16.cu,
// paged_attn_bf16_e4m3.cu, paged_attn_f16_e4m3.cu).
//
// out = softmax(scale q K^T) V for the query heads that share a kv head.  The
// cache's keys and values are read once, so the kernel should be bound by
// memory; the arithmetic (4 flops per cache element and query head) runs on
// warp-level matrix instructions.  Their 16-row side holds what there is much
// of -- positions in S^T = K Q^T, head elements in O^T = V^T P^T -- and their
// 8-column side the query heads, so up to eight shared heads waste nothing; the
// heads as the 16 rows would take twice the instructions a step.
//
// GB300 (one device to the next 2% apart): two sequences of 130,001 and 131,072
// positions, 8 kv heads of 128 and 64 query heads: 184 to 188 us for 1.07 GB,
// 5.7 to 5.8 TB/s, 84 to 86% of a plain copy's rate (with the arithmetic left out
// 178: the loads, and SMs that do not finish together, are the bound).  64
// sequences of 0 to 8192 positions, 32 query heads: 49.5 to 50.7 us for 253 MB,
// 5.0 to 5.1 TB/s; some 11 us of it are the start (list of lengths, page
// numbers, the first rows) and the ends of segments, and moderate batches pay
// the same: 4 sequences of 2000 13.5 us at a floor of 4.8, 16 of 100 to 4000
// 21.9 at 10.9.  E4M3 caches: short rows are bound by the conversions'
// instructions (33 windows of up to 2001 positions, 4 kv heads of 80: 19.1 us
// for 36 MB; 64 sequences of 100 to 8192, 8 kv heads of 64: 36.7 at a floor of
// 18.2, of 80: 50 to 57 at 23); long ones by their loads (two sequences of
// 100,000, 8 kv heads of 128: 80 to 85 us for 410 MB, and 82 of 85 with the
// arithmetic left out, 5.0 TB/s; the 16-bit cache of the same positions 140 us
// for 820 MB, 5.9 TB/s).
//
// Nine to 16 query heads a kv head take two tiles of heads, in 217 to 255
// registers: 16 sequences of 100 to 8192, 4 kv heads of 128 with 16 query heads
// each, 40 us at a floor of 9.7.  Heads of 256 with two tiles spill (416 to 472
// bytes stored a thread): 64 such sequences, 2 kv heads, 92 us at 36.5, where
// one tile takes 55.  Head sizes from 136 to 248 run as 256, one CTA an SM: 8
// kv heads of 192 133 us at 109, of 136 135 at 77.
//
// Work.  A segment is one (sequence, kv head, group of 8 or 16 query heads);
// its positions are cut into tiles of four warps' steps.  All segments' tiles,
// laid end to end with kAttnSegmentCost empty units before each segment (what
// starting and ending one costs), are cut into equal contiguous ranges, one
// per CTA of a grid that fills the device once, so ragged lengths balance
// without any host knowledge of them and a long cache is split as often as the
// device needs.  A CTA that holds a whole segment writes its output; otherwise
// it leaves (m, l, O) in the workspace, and the last of the segment's CTAs to
// arrive (a counter, no waiting) joins them in the order of the positions, so
// results do not depend on timing.
//
// Inside a CTA each of four warps takes its own positions of every tile (16,
// or 32 where rows are short): its own copy pipeline (no block barrier), its
// own running maximum and sum, joined with the other warps' at the segment's
// end in the pipeline slots just consumed.  The copies run ahead across segment
// ends.  More and smaller ranges than one per resident CTA cost more in starts
// than they balance (the long sequences in twice as many: 213 us).  Rows of K and V lie in shared memory at an
// odd number of 16-byte chunks apart, so the eight rows of a matrix load fall
// into different banks.
#pragma once

#include <cfloat>
#include <climits>

#include <cuda_runtime.h>

#include "common.cuh"
#include "elem.cuh"
#include "paged_attn_host.h"
#include "serving.h"
#include "serving_host.h"

namespace dgb {

__host__ __device__ constexpr int next_pow2(int v) { return v <= 1 ? 1 : 2 * next_pow2((v + 1) / 2); }

// KD: 16-element blocks of a head; NH: 8-head tiles of a segment.
template <int KD, bool FP8, int NH>
struct AttnShape {
    static constexpr int kHeads = 8 * NH;
    // CTAs an SM holds, and steps in the pipeline of a warp.  E4M3 rows of up to 80 bytes: a step's instructions (the
    // conversions), not its bytes, are the longer part, and more warps count for more than a deeper pipeline: 64 sequences
    // of 100 to 8192 positions, 8 kv heads of 64, took 36.4 us so and 40.1 with two CTAs and three stages; longer rows
    // want the loads in flight (two sequences of 100,000, heads of 128: 92.4 so and 87.4).
    static constexpr bool kManyCtas = FP8 && NH == 1 && KD <= 5;
    static constexpr int kCtas = kManyCtas ? 3 : (KD <= 8 ? 2 : 1);
    static constexpr int kStages = kManyCtas ? 2 : 3;
    static constexpr int kDim = KD * 16;                 // head elements held (head_dim rounded up)
    static constexpr int kBytes = FP8 ? 1 : 2;
    static constexpr int kChunks = KD * kBytes;          // 16-byte chunks of a row
    static constexpr int kTokens = kChunks <= 8 || FP8 ? 32 : 16;   // positions of one warp's step
    static constexpr int kTile = kAttnWarps * kTokens;
    static constexpr int kPitch = (kChunks | 1) * 16;    // bytes between rows
    static constexpr int kRowsBytes = kTokens * kPitch;
    static constexpr int kMergePitch = kDim + 4;         // floats; a slot also takes one warp's O at a segment's end
    static constexpr int kMergeBytes = kHeads * kMergePitch * 4;
    static constexpr int kStageBytes = 2 * kRowsBytes > kMergeBytes ? 2 * kRowsBytes : kMergeBytes;
    static constexpr int kRingBytes = kAttnWarps * kStages * kStageBytes;
    static constexpr int kAddrBytes = kAttnWarps * kTokens * 16;
    static constexpr int kSmemBytes = kRingBytes + kAddrBytes;
    static constexpr int kSlotFloats = kHeads * (kDim + 2);   // one partial: O, m, l
    // copies: a power of two of lanes per row
    static constexpr int kLanesPerRow = next_pow2(kChunks);
    static constexpr int kRowsPerCopy = 32 / kLanesPerRow;
    static constexpr int kCopies = kTokens / kRowsPerCopy;
};

// Position in the list of all tiles: tile `tile` of `tiles` of segment (b, hv), `left` units before the range's end.
struct TileWalk {
    int b, hv, tile, tiles, first, length;   // positions [first, length)
    int64_t left;                            // > 0: this tile belongs to the range
};

__device__ __forceinline__ void sequence_span(const AttnParams& p, int b, int& first, int& length) {
    const int64_t most = (int64_t)p.a.table_width * p.page_size;
    length = max(0, p.a.lengths[b]);
    if (length > most) length = (int)most;
    first = p.window > 0 ? max(0, length - p.window) : 0;
}
template <int TILE>
__device__ __forceinline__ int tiles_of(int first, int length) {
    return (int)(((uint32_t)(length - first) + (TILE - 1)) / TILE);
}

template <typename T, typename TQ, bool FP8, int KD, int NH>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<KD, FP8, NH>::kCtas) paged_attn_kernel(const __grid_constant__ AttnParams p) {
    using S = AttnShape<KD, FP8, NH>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan_part[kAttnWarps];
    __shared__ int found_b;
    __shared__ int64_t found_rest;
    __shared__ float warp_m[kAttnWarps][S::kHeads], warp_l[kAttnWarps][S::kHeads];
    __shared__ uint32_t stage_mask[kAttnWarps][S::kStages];
    __shared__ int join_now;
    constexpr int kTokens = S::kTokens;
    constexpr uint32_t kFull = kTokens == 32 ? 0xFFFFFFFFu : 0xFFFFu;
    // Probabilities are held times 2^kShift, which O and l share.  As f16 operands they keep their 11 bits down to 2^-29 that
    // way (2^-14 without); 2^15 is the largest power whose probability of one is a finite f16.
    constexpr float kShift = std::is_same<T, __half>::value ? 15.f : 0.f;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, j4 = lane & 3;
    const int HV = p.segments_per_sequence;
    const int B = p.a.batch;
    uint8_t* ring = smem + (size_t)warp * S::kStages * S::kStageBytes;
    longlong2* addr = reinterpret_cast<longlong2*>(smem + S::kRingBytes) + warp * kTokens;
    const int row_chunks = p.head_dim * S::kBytes / 16;
    if (row_chunks < S::kChunks) {
        // chunks past head_dim are never copied: zeros, for the products that run over them
        for (int i = threadIdx.x; i < S::kRingBytes / 16; i += kAttnThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    griddep_wait();
    griddep_launch_dependents();

    auto out_row = [&](int b, int head) { return static_cast<TQ*>(p.a.out) + b * p.a.out_batch + head * p.a.out_head; };
    auto write_empty = [&]() {      // outputs of sequences without a visible position
        for (int b = blockIdx.x; b < B; b += gridDim.x) {
            int first, length;
            sequence_span(p, b, first, length);
            if (length > first) continue;
            for (int i = threadIdx.x; i < p.heads * (p.head_dim / 2); i += kAttnThreads) {
                const int h = i / (p.head_dim / 2);
                reinterpret_cast<uint32_t*>(out_row(b, h))[i - h * (p.head_dim / 2)] = 0u;
            }
            if (p.a.lse)
                for (int h = threadIdx.x; h < p.heads; h += kAttnThreads) p.a.lse[(int64_t)b * p.heads + h] = -INFINITY;
        }
    };

    // ---------------------------------------------------------------- this CTA's range of tiles
    auto units_of = [&](int b) -> int64_t {      // of one sequence
        int first, length;
        if (b >= B) return 0;
        sequence_span(p, b, first, length);
        const int t = tiles_of<S::kTile>(first, length);
        return t > 0 ? (int64_t)(t + kAttnSegmentCost) * HV : 0;
    };
    // Units before this thread's sequence among 128 of them, and all of them's.
    auto scan = [&](int64_t v, int64_t& all) {
        int64_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();
        if (lane == 31) scan_part[warp] = incl;
        __syncthreads();
        int64_t lo = incl - v;
        all = 0;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w < warp) lo += scan_part[w];
            all += scan_part[w];
        }
        return lo;
    };
    int64_t v = units_of(threadIdx.x), all;
    int64_t lo = scan(v, all);                   // the first 128 sequences
    int64_t total = all;
    if (B > kAttnThreads) {
        int64_t rest = 0;
        for (int b = threadIdx.x + kAttnThreads; b < B; b += kAttnThreads) rest += units_of(b);
        int64_t more;
        scan(rest, more);
        total += more;
    }
    // Small problems leave CTAs idle rather than cut segments finely.
    const int ctas = (int)min((int64_t)gridDim.x, (total + kAttnMinUnits - 1) / kAttnMinUnits);
    if ((int)blockIdx.x >= ctas) {
        write_empty();
        return;
    }
    auto range_start = [&](int c) { return total * c / ctas; };
    const int64_t range0 = range_start(blockIdx.x), range1 = range_start(blockIdx.x + 1);
    // The sequence that holds unit range0: 128 sequences at a time.
    int64_t before = 0;
    for (int base = 0;;) {
        if (range0 >= before + lo && range0 < before + lo + v) {
            found_b = base + threadIdx.x;
            found_rest = range0 - before - lo;
        }
        before += all;
        base += kAttnThreads;
        if (before > range0 || base >= B) break;
        v = units_of(base + threadIdx.x);
        lo = scan(v, all);
    }
    __syncthreads();

    TileWalk at;      // the step being computed
    at.b = found_b;
    sequence_span(p, at.b, at.first, at.length);
    at.tiles = tiles_of<S::kTile>(at.first, at.length);
    const int per_segment = at.tiles + kAttnSegmentCost;
    at.hv = found_rest <= INT_MAX ? (int)found_rest / per_segment : (int)(found_rest / per_segment);
    at.tile = (int)(found_rest - (int64_t)at.hv * per_segment) - kAttnSegmentCost;
    at.left = range1 - range0;
    int64_t unit = range0;           // of the step being computed
    if (at.tile < 0) {               // the range starts with (part of) a segment's empty units
        at.left += at.tile;
        unit -= at.tile;
        at.tile = 0;
    }
    TileWalk ahead = at;             // the step whose addresses are fetched next
    auto advance = [&](TileWalk& w) {
        --w.left;
        if (++w.tile < w.tiles) return;
        w.left -= kAttnSegmentCost;
        w.tile = 0;
        if (++w.hv < HV) return;
        w.hv = 0;
        do {
            if (++w.b >= B) {        // past the last tile
                w.left = 0;
                return;
            }
            sequence_span(p, w.b, w.first, w.length);
            w.tiles = tiles_of<S::kTile>(w.first, w.length);
        } while (w.tiles == 0);
    };

    // ---------------------------------------------------------------- copies
    // Lane r fetches the page of its row r of the next step; the number is used one step later.
    const int copy_row = lane / S::kLanesPerRow, copy_chunk = lane % S::kLanesPerRow;
    const bool copies = copy_chunk < row_chunks;
    const uint32_t copy_dst = smem_u32(ring) + copy_row * S::kPitch + copy_chunk * 16;
    const uint8_t* kbase = static_cast<const uint8_t*>(p.a.k_cache) + copy_chunk * 16;
    const uint8_t* vbase = static_cast<const uint8_t*>(p.a.v_cache) + copy_chunk * 16;
    const int64_t k_place = p.a.k_place * S::kBytes, v_place = p.a.v_place * S::kBytes;
    struct Next {
        int page, place, head;
        bool live;
    };
    auto fetch = [&]() {
        Next next;
        next.live = ahead.left > 0;
        next.page = -1;
        next.place = next.head = 0;
        if (!next.live) return next;
        const uint32_t pos = (uint32_t)ahead.first + (uint32_t)ahead.tile * S::kTile + warp * kTokens + (lane & (kTokens - 1));
        next.head = ahead.hv / p.head_groups;
        if (pos < (uint32_t)ahead.length) {
            const int col = p.page_shift >= 0 ? (int)(pos >> p.page_shift) : (int)(pos / (uint32_t)p.page_size);
            next.place = (int)pos - col * p.page_size;
            next.page = p.a.block_table[ahead.b * p.a.table_stride + col];
        }
        advance(ahead);
        return next;
    };
    auto issue = [&](const Next& next, int stage) {
        const int next_page = next.page, next_place = next.place, next_head = next.head;
        if (next.live) {
            const bool have = next_page >= 0 && next_page < p.a.num_pages;
            const int page0 = __shfl_sync(0xffffffffu, next_page, 0), first_place = __shfl_sync(0xffffffffu, next_place, 0);
            const uint32_t mask = __ballot_sync(0xffffffffu, have) & kFull;
            if (lane == 0) stage_mask[warp][stage] = mask;
            const uint32_t dst = copy_dst + stage * S::kStageBytes;
            // The places have to follow one another too: neighbouring columns of the block table may name the same page.
            const bool in_line = next_page == page0 && next_place == first_place + (lane & (kTokens - 1));
            if (mask == kFull && __all_sync(0xffffffffu, in_line)) {
                // one column's page holds all rows (the common case): they lie one place stride apart
                const int64_t place0 = first_place + copy_row;
                const uint8_t* kp = kbase + (page0 * p.a.k_page + next_head * p.a.k_head) * S::kBytes + place0 * k_place;
                const uint8_t* vp = vbase + (page0 * p.a.v_page + next_head * p.a.v_head) * S::kBytes + place0 * v_place;
                if (copies) {
#pragma unroll
                    for (int i = 0; i < S::kCopies; ++i) {
                        cp_async_16(dst + i * S::kRowsPerCopy * S::kPitch, kp);
                        cp_async_16(dst + i * S::kRowsPerCopy * S::kPitch + S::kRowsBytes, vp);
                        kp += S::kRowsPerCopy * k_place;
                        vp += S::kRowsPerCopy * v_place;
                    }
                }
            } else if (mask) {
                // rows on several pages, or past the end (those become zeros)
                if (lane < kTokens) {
                    const int64_t pg = have ? next_page : 0, pl = have ? next_place : 0;
                    longlong2 o;
                    o.x = (pg * p.a.k_page + next_head * p.a.k_head) * S::kBytes + pl * k_place;
                    o.y = (pg * p.a.v_page + next_head * p.a.v_head) * S::kBytes + pl * v_place;
                    addr[lane] = o;
                }
                __syncwarp();
                if (copies) {
#pragma unroll
                    for (int i = 0; i < S::kCopies; ++i) {
                        const int row = copy_row + i * S::kRowsPerCopy;
                        const longlong2 o = addr[row];
                        const uint32_t bytes = (mask >> row) & 1u ? 16u : 0u;
                        cp_async_16_zfill(dst + i * S::kRowsPerCopy * S::kPitch, kbase + o.x, bytes);
                        cp_async_16_zfill(dst + i * S::kRowsPerCopy * S::kPitch + S::kRowsBytes, vbase + o.y, bytes);
                    }
                }
            }
        }
        cp_async_commit();
        __syncwarp();
    };

    // ---------------------------------------------------------------- state of the running softmax
    // O^T: o[n][blk], heads n * 8 + 2 j4 and + 1 (elements 0, 2 and 1, 3), dims of block blk: quad and quad + 8 (elements 0, 1
    // and 2, 3), or 2 quad and 2 quad + 1 for E4M3 caches.  m, l: of the same two heads of each tile.
    uint32_t q[NH][KD][2];
    float o[NH][KD][4];
    float m[NH][2], l[NH][2];
    float sc[NH][2];                                          // score -> log2 units
    int rows = 0, head0 = 0;                                  // the segment's query heads
    bool first_segment = true;

    auto load_query = [&]() {
        const int kvh = at.hv / p.head_groups, hg = at.hv - kvh * p.head_groups;
        head0 = kvh * p.group + hg * S::kHeads;
        rows = min(S::kHeads, p.group - hg * S::kHeads);
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const TQ* row = static_cast<const TQ*>(p.a.q) + at.b * p.a.q_batch + (int64_t)(head0 + n * 8 + quad) * p.a.q_head;
            const bool in = n * 8 + quad < rows;
#pragma unroll
            for (int kk = 0; kk < KD; ++kk) {
                // the two element pairs of this lane: (2j, 2j+1) and (2j+8, 2j+9), or, for E4M3 caches, four neighbours
                // (the product's order over the head dimension is free; see the key fragments)
                const int da = kk * 16 + (FP8 ? 4 * j4 : 2 * j4), db = FP8 ? da + 2 : da + 8;
                q[n][kk][0] = in && da < p.head_dim ? *reinterpret_cast<const uint32_t*>(row + da) : 0u;
                q[n][kk][1] = in && db < p.head_dim ? *reinterpret_cast<const uint32_t*>(row + db) : 0u;
            }
        }
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            sc[n][0] = sc[n][1] = p.score_log2;
            if (p.negate) {
#pragma unroll
                for (int kk = 0; kk < KD; ++kk) {
                    q[n][kk][0] ^= 0x80008000u;
                    q[n][kk][1] ^= 0x80008000u;
                }
            }
            if constexpr (FP8 && !std::is_same<T, TQ>::value) {
                // bf16 queries against f16 keys: each head is scaled by a power of two to a largest element in [1, 2)
                // (exact; elements 2^-14 of the largest and smaller lose bits) and its scores are scaled back
                float top = 0.f;
#pragma unroll
                for (int kk = 0; kk < KD; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = unpack2<TQ>(q[n][kk][i]);
                        top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
#pragma unroll
                for (int s = 1; s < 4; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                // biased exponent, kept where 2^e and 2^-e are normal numbers
                const int e = min(max((int)(__float_as_uint(top) >> 23), 1), 252);
                const float down = __uint_as_float((uint32_t)(254 - e) << 23);
                const float up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
                for (int kk = 0; kk < KD; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = unpack2<TQ>(q[n][kk][i]);
                        q[n][kk][i] = round2<T>(v.x * down, v.y * down);
                    }
                // this lane loaded head quad and scales scores of heads 2 j4 and 2 j4 + 1
                sc[n][0] = fmaxf(sc[n][0] * __shfl_sync(0xffffffffu, up, 8 * j4), FLT_MIN);
                sc[n][1] = fmaxf(sc[n][1] * __shfl_sync(0xffffffffu, up, 8 * j4 + 4), FLT_MIN);
            }
#pragma unroll
            for (int blk = 0; blk < KD; ++blk)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][blk][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = -FLT_MAX;
                l[n][i] = 0.f;
            }
        }
    };

    auto compute = [&](int stage) {
        const uint32_t mask = stage_mask[warp][stage];
        if (!mask) return;
        const uint32_t ks = smem_u32(ring + (size_t)stage * S::kStageBytes), vs = ks + S::kRowsBytes;
        constexpr int kT = kTokens / 16;        // 16-position row tiles of S^T
        float s[NH][kT][4];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            // two accumulators: the chains of dependent products are half as long
            float x[NH][4] = {}, y[NH][4] = {};
            if constexpr (FP8) {
                // One 32-bit word of a lane is four neighbouring elements of its row: two f16 pairs, the two k halves of one
                // step.  A load covers two 16-element blocks.
                const uint32_t base = ks + (t * 16 + (lane & 15)) * S::kPitch;
#pragma unroll
                for (int kk = 0; kk < KD; kk += 2) {
                    uint32_t r[4];
                    ldmatrix_x4(base + (kk + (kk + 1 < KD ? (lane >> 4) : 0)) * 16, r);
                    const uint32_t a0[4] = {e4m3x2_to_half2(r[0]), e4m3x2_to_half2(r[1]), e4m3x2_to_half2(r[0] >> 16),
                                            e4m3x2_to_half2(r[1] >> 16)};
#pragma unroll
                    for (int n = 0; n < NH; ++n) mma_16816<T>(x[n], a0, q[n][kk][0], q[n][kk][1]);
                    if (kk + 1 < KD) {
                        const uint32_t a1[4] = {e4m3x2_to_half2(r[2]), e4m3x2_to_half2(r[3]), e4m3x2_to_half2(r[2] >> 16),
                                                e4m3x2_to_half2(r[3] >> 16)};
#pragma unroll
                        for (int n = 0; n < NH; ++n) mma_16816<T>(y[n], a1, q[n][kk + 1][0], q[n][kk + 1][1]);
                    }
                }
            } else {
                const uint32_t base = ks + (t * 16 + (lane & 15)) * S::kPitch + (lane >> 4) * 16;
#pragma unroll
                for (int kk = 0; kk < KD; ++kk) {
                    uint32_t a[4];
                    ldmatrix_x4(base + kk * 32, a);
#pragma unroll
                    for (int n = 0; n < NH; ++n) mma_16816<T>(kk & 1 ? y[n] : x[n], a, q[n][kk][0], q[n][kk][1]);
                }
            }
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][t][i] = x[n][i] + y[n][i];
        }
        if (mask != kFull) {
#pragma unroll
            for (int t = 0; t < kT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (!((mask >> (t * 16 + quad + 8 * h)) & 1u)) {
#pragma unroll
                        for (int n = 0; n < NH; ++n) s[n][t][2 * h] = s[n][t][2 * h + 1] = -INFINITY;
                    }
        }
        // Running maxima in log2 units (the scales sc are positive, see load_query).
        float top[NH][2];
        bool grows = false;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = fmaxf(s[n][0][i], s[n][0][2 + i]);
#pragma unroll
                for (int t = 1; t < kT; ++t) v = fmaxf(v, fmaxf(s[n][t][i], s[n][t][2 + i]));
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                top[n][i] = v * sc[n][i];
                grows |= top[n][i] > m[n][i];
            }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float fresh = fmaxf(m[n][i], top[n][i]);
                    const float f = exp2_fast(m[n][i] - fresh);
                    m[n][i] = fresh;
                    l[n][i] *= f;
#pragma unroll
                    for (int blk = 0; blk < KD; ++blk) {
                        o[n][blk][i] *= f;
                        o[n][blk][2 + i] *= f;
                    }
                }
        }
        // Probabilities times 2^kShift, as the 16-bit right operand P^T of the product with V (the matrix instruction takes
        // 16-bit operands); their sum l is taken in fp32 before that rounding, O stays fp32.
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            uint32_t b[NH][2];
#pragma unroll
            for (int n = 0; n < NH; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][t][i] = exp2_fast(fmaf(s[n][t][i], sc[n][i & 1], kShift - m[n][i & 1]));
                l[n][0] += s[n][t][0] + s[n][t][2];
                l[n][1] += s[n][t][1] + s[n][t][3];
                b[n][0] = transpose_8x8(round2<T>(s[n][t][0], s[n][t][1]));
                b[n][1] = transpose_8x8(round2<T>(s[n][t][2], s[n][t][3]));
            }
            if constexpr (FP8) {
                // a transposed load moves pairs of elements: bytes (t0 d0, t0 d1, t1 d0, t1 d1); reordered to pairs of
                // positions, a 16-element block's even elements are rows 0..7 of its tile and its odd ones rows 8..15
                const uint32_t base = vs + (t * 16 + (lane & 15)) * S::kPitch;
                auto tile = [&](int blk, uint32_t lo, uint32_t hi) {
                    const uint32_t u = __byte_perm(lo, 0u, 0x3120), v = __byte_perm(hi, 0u, 0x3120);
                    const uint32_t a[4] = {e4m3x2_to_half2(u), e4m3x2_to_half2(u >> 16), e4m3x2_to_half2(v), e4m3x2_to_half2(v >> 16)};
#pragma unroll
                    for (int n = 0; n < NH; ++n) mma_16816<T>(o[n][blk], a, b[n][0], b[n][1]);
                };
#pragma unroll
                for (int blk = 0; blk < KD; blk += 2) {
                    uint32_t r[4];
                    // the last odd block loads its own chunk twice
                    ldmatrix_x4_trans(base + (blk + (blk + 1 < KD ? (lane >> 4) : 0)) * 16, r);
                    tile(blk, r[0], r[1]);
                    if (blk + 1 < KD) tile(blk + 1, r[2], r[3]);
                }
            } else {
                const uint32_t base = vs + (t * 16 + (lane & 7) + (lane >> 4) * 8) * S::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
                for (int blk = 0; blk < KD; ++blk) {
                    uint32_t a[4];
                    ldmatrix_x4_trans(base + blk * 32, a);
#pragma unroll
                    for (int n = 0; n < NH; ++n) mma_16816<T>(o[n][blk], a, b[n][0], b[n][1]);
                }
            }
        }
    };

    constexpr float kLn2 = 0.693147180559945309f;
    auto write_lse = [&](int b, int row, float m, float l) {
        if (p.a.lse) p.a.lse[(int64_t)b * p.heads + head0 + row] = l > 0.f || l != l ? (m + (log2f(l) - kShift)) * kLn2 : -INFINITY;
    };

    // The segment's positions of this CTA are done: join the warps, then write or leave a partial.  Each warp lays its O
    // into the pipeline slot it just consumed (free until the next copies are issued).
    auto flush = [&](int stage) {
        float* own = reinterpret_cast<float*>(ring + (size_t)stage * S::kStageBytes);
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = n * 8 + 2 * j4 + i;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], d);
                if (quad == 0) {
                    warp_m[warp][r] = m[n][i];
                    warp_l[warp][r] = l[n][i];
                }
                if (r < rows) {
#pragma unroll
                    for (int blk = 0; blk < KD; ++blk) {
                        const int d = blk * 16 + (FP8 ? 2 * quad : quad);
                        own[r * S::kMergePitch + d] = o[n][blk][i];
                        own[r * S::kMergePitch + d + (FP8 ? 1 : 8)] = o[n][blk][2 + i];
                    }
                }
            }
        __syncthreads();
        auto joined = [&](int r, int d, float& m, float& l) {     // four columns of a row, over the warps in order
            m = -FLT_MAX;
            l = 0.f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, warp_m[w][r]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float f = exp2_fast(warp_m[w][r] - m);
                const float4 x = *reinterpret_cast<const float4*>(smem + ((size_t)w * S::kStages + stage) * S::kStageBytes +
                                                                  (r * S::kMergePitch + d) * 4);
                l = fmaf(warp_l[w][r], f, l);
                v.x = fmaf(x.x, f, v.x);
                v.y = fmaf(x.y, f, v.y);
                v.z = fmaf(x.z, f, v.z);
                v.w = fmaf(x.w, f, v.w);
            }
            return v;
        };
        const int64_t seg0 = unit - at.tile, seg1 = seg0 + at.tiles;   // the segment's tiles, as units
        const int quarter = p.head_dim / 4;
        // the CTAs that share the segment: those of its first and last tile and all between
        const bool whole = seg0 >= range0 && seg1 <= range1;
        if (whole) {
            for (int i = threadIdx.x; i < rows * quarter; i += kAttnThreads) {
                const int r = i / quarter, d = (i - r * quarter) * 4;
                float m, l;
                const float4 v = joined(r, d, m, l);
                const float f = l > 0.f || l != l ? p.a.v_scale / l : 0.f;
                *reinterpret_cast<uint2*>(out_row(at.b, head0 + r) + d) =
                    make_uint2(round2<TQ>(v.x * f, v.y * f), round2<TQ>(v.z * f, v.w * f));
                if (d == 0) write_lse(at.b, r, m, l);
            }
            __syncthreads();
            return;
        }
        float* slot = p.partials + ((int64_t)blockIdx.x * 2 + (first_segment ? 0 : 1)) * S::kSlotFloats;
        for (int i = threadIdx.x; i < rows * quarter; i += kAttnThreads) {
            const int r = i / quarter, d = (i - r * quarter) * 4;
            float m, l;
            __stcg(reinterpret_cast<float4*>(slot + r * S::kDim + d), joined(r, d, m, l));
            if (d == 0) {
                __stcg(slot + S::kHeads * S::kDim + r, m);
                __stcg(slot + S::kHeads * (S::kDim + 1) + r, l);
            }
        }
        const int c0 = (int)(((seg0 + 1) * ctas - 1) / total), c1 = (int)((seg1 * ctas - 1) / total);
        uint32_t* counter = p.counters + (int64_t)at.b * HV + at.hv;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) join_now = atomicAdd(counter, 1u) == (uint32_t)(c1 - c0);
        __syncthreads();
        if (join_now) {
            __threadfence();
            // the first CTA's other slot, if it ended another segment before this one
            const bool c0_first = range_start(c0) >= seg0 - kAttnSegmentCost;
            auto slot_of = [&](int c) {
                return p.partials + ((int64_t)c * 2 + (c == c0 && !c0_first ? 1 : 0)) * S::kSlotFloats;
            };
            for (int i = threadIdx.x; i < rows * quarter; i += kAttnThreads) {
                const int r = i / quarter, d = (i - r * quarter) * 4;
                // eight partials' loads at a time
                constexpr int kMany = 8;
                float M = -FLT_MAX, L = 0.f;
                for (int c = c0; c <= c1; c += kMany) {
                    float x[kMany];
#pragma unroll
                    for (int u = 0; u < kMany; ++u) x[u] = __ldcg(slot_of(min(c + u, c1)) + S::kHeads * S::kDim + r);
#pragma unroll
                    for (int u = 0; u < kMany; ++u) M = fmaxf(M, x[u]);
                }
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = c0; c <= c1; c += kMany) {
                    float pm[kMany], pl[kMany];
                    float4 x[kMany];
#pragma unroll
                    for (int u = 0; u < kMany; ++u) {
                        const float* sl = slot_of(min(c + u, c1));
                        pm[u] = __ldcg(sl + S::kHeads * S::kDim + r);
                        pl[u] = __ldcg(sl + S::kHeads * (S::kDim + 1) + r);
                        x[u] = __ldcg(reinterpret_cast<const float4*>(sl + r * S::kDim + d));
                    }
#pragma unroll
                    for (int u = 0; u < kMany; ++u) {
                        if (c + u > c1) break;
                        const float f = exp2_fast(pm[u] - M);
                        L = fmaf(pl[u], f, L);
                        v.x = fmaf(x[u].x, f, v.x);
                        v.y = fmaf(x[u].y, f, v.y);
                        v.z = fmaf(x[u].z, f, v.z);
                        v.w = fmaf(x[u].w, f, v.w);
                    }
                }
                const float f = L > 0.f || L != L ? p.a.v_scale / L : 0.f;
                *reinterpret_cast<uint2*>(out_row(at.b, head0 + r) + d) =
                    make_uint2(round2<TQ>(v.x * f, v.y * f), round2<TQ>(v.z * f, v.w * f));
                if (d == 0) write_lse(at.b, r, M, L);
            }
            if (threadIdx.x == 0) *counter = 0u;     // ready for the next launch
        }
        __syncthreads();
    };

    // ---------------------------------------------------------------- the loop
    Next next;
    {
        // the first steps' page numbers and the first query are fetched together
        Next begin[S::kStages];
#pragma unroll
        for (int i = 0; i < S::kStages; ++i) begin[i] = fetch();
        if (at.left > 0) load_query();
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) issue(begin[i], i);
        next = begin[S::kStages - 1];
    }
    int stage = 0, fill = S::kStages - 1;
    while (at.left > 0) {
        cp_async_wait<S::kStages - 2>();
        __syncwarp();
        issue(next, fill);        // the slot computed on in the previous step
        next = fetch();
        compute(stage);
        if (at.tile + 1 == at.tiles || at.left == 1) {
            flush(stage);
            if (row_chunks < S::kChunks) {      // O went over the zeros behind head_dim
                const int pad = S::kChunks - row_chunks;
                for (int i = lane; i < kTokens * pad; i += 32)
                    *reinterpret_cast<uint4*>(ring + (size_t)stage * S::kStageBytes + (i / pad) * S::kPitch + (row_chunks + i % pad) * 16) =
                        make_uint4(0, 0, 0, 0);
                __syncwarp();
            }
            first_segment = false;
            const int64_t left = at.left;
            advance(at);
            unit += left - at.left;
            if (at.left > 0) load_query();
        } else {
            ++at.tile;
            --at.left;
            ++unit;
        }
        if (++stage == S::kStages) stage = 0;
        if (++fill == S::kStages) fill = 0;
    }
    cp_async_wait<0>();
    write_empty();
}

template <typename T, typename TQ, bool FP8, int KD, int NH>
cudaError_t attn_launch(const AttnParams& p, int grid, cudaStream_t stream) {
    return launch_dependent(paged_attn_kernel<T, TQ, FP8, KD, NH>, dim3((unsigned)grid), dim3(kAttnThreads),
                            AttnShape<KD, FP8, NH>::kSmemBytes, stream, p);
}

// Raises the kernel's shared-memory limit and says how many CTAs an SM holds.
template <typename T, typename TQ, bool FP8, int KD, int NH>
cudaError_t attn_prepare(AttnVariant* v) {
    using S = AttnShape<KD, FP8, NH>;
    auto kern = paged_attn_kernel<T, TQ, FP8, KD, NH>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
    if (e != cudaSuccess) return e;
    v->smem_bytes = S::kSmemBytes;
    v->slot_floats = S::kSlotFloats;
    v->tile_tokens = S::kTile;
    v->heads = S::kHeads;
    v->launch = &attn_launch<T, TQ, FP8, KD, NH>;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v->ctas_per_sm, kern, kAttnThreads, S::kSmemBytes);
}

// The head sizes held: head_dim is rounded up to one of them.  Up to eight query heads a kv head take one 8-head tile.
template <typename T, typename TQ, bool FP8, int NH>
cudaError_t attn_variant_heads(int head_dim, AttnVariant* v) {
    if (head_dim <= 64) return attn_prepare<T, TQ, FP8, 4, NH>(v);
    if (head_dim <= 80) return attn_prepare<T, TQ, FP8, 5, NH>(v);
    if (head_dim <= 96) return attn_prepare<T, TQ, FP8, 6, NH>(v);
    if (head_dim <= 128) return attn_prepare<T, TQ, FP8, 8, NH>(v);
    return attn_prepare<T, TQ, FP8, 16, NH>(v);
}
template <typename T, typename TQ, bool FP8>
cudaError_t attn_variant(int head_dim, int group, AttnVariant* v) {
    return group <= 8 ? attn_variant_heads<T, TQ, FP8, 1>(head_dim, v) : attn_variant_heads<T, TQ, FP8, 2>(head_dim, v);
}

}  // namespace dgb
