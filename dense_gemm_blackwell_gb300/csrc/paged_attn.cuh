// paged_attn.cuh -- attention of one new token per sequence over a paged
// key-value cache (include/serving.h): kernel and launcher, one translation
// unit per pair of query and cache types (paged_attn_bf16.cu, paged_attn_f16.cu,
// paged_attn_bf16_e4m3.cu, paged_attn_f16_e4m3.cu).
//
// out = softmax(scale q K^T) V for the query heads that share a kv head.  The
// cache's keys and values are read once, so the kernel is bound by memory; the
// arithmetic (4 flops per cache element and query head) is kept off the
// critical path by warp-level matrix instructions with the shared query heads
// as the 16 rows of the tile.
//
// Work.  A segment is one (sequence, kv head, group of up to 16 query heads);
// its positions are cut into tiles of 64.  All segments' tiles, laid end to
// end, are cut into equal contiguous ranges, one per CTA of a grid that fills
// the device once, so ragged lengths balance without any host knowledge of
// them and a long cache is split as often as the device needs.  A CTA that
// holds a whole segment writes its output; otherwise it leaves (m, l, O) in
// the workspace, and the last of the segment's CTAs to arrive (a counter, no
// waiting) joins them in the order of the positions, so results do not depend
// on timing.
//
// Inside a CTA each of four warps takes 16 positions of every tile on its own:
// its own copy pipeline (kStages deep, no block barrier), its own running
// maximum and sum, joined with the other warps' at the segment's end.  The
// copies run ahead across segment ends.  Rows of K and V lie in shared memory
// at an odd number of 16-byte chunks apart, so the eight rows of a matrix load
// fall into different banks.
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

template <int KD, bool FP8>
struct AttnShape {
    static constexpr int kDim = KD * 16;                 // head elements held (head_dim rounded up)
    static constexpr int kChunks = FP8 ? KD : 2 * KD;    // 16-byte chunks of a row
    static constexpr int kPitch = (kChunks | 1) * 16;    // bytes between rows
    static constexpr int kRowsBytes = kAttnWarpTokens * kPitch;
    static constexpr int kStageBytes = 2 * kRowsBytes;   // one warp's keys and values of one step
    static constexpr int kMergePitch = kDim + 4;         // floats
    static constexpr int kRingBytes = kAttnWarps * kAttnStages * kStageBytes;
    static constexpr int kAddrBytes = kAttnWarps * kAttnWarpTokens * 16;
    static constexpr int kMergeBytes = 16 * kMergePitch * 4;
    static constexpr int kSmemBytes = kRingBytes + kAddrBytes + kMergeBytes;
    static constexpr int kSlotFloats = 16 * kDim + 32;   // one partial: O, m, l
};

// Position in the list of all tiles: tile `tile` of `tiles` of segment (b, hv).
struct TileWalk {
    int b, hv, tile, tiles, first, length;   // positions [first, length)
};

__device__ __forceinline__ void sequence_span(const AttnParams& p, int b, int& first, int& length) {
    const int64_t most = (int64_t)p.a.table_width * p.page_size;
    length = max(0, p.a.lengths[b]);
    if (length > most) length = (int)most;
    first = p.window > 0 ? max(0, length - p.window) : 0;
}
__device__ __forceinline__ int tiles_of(int first, int length) {
    return (int)(((int64_t)length - first + kAttnTile - 1) / kAttnTile);
}

template <typename T, typename TQ, bool FP8, int KD>
__global__ void __launch_bounds__(kAttnThreads, KD <= 8 ? 2 : 1) paged_attn_kernel(const __grid_constant__ AttnParams p) {
    using S = AttnShape<KD, FP8>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan_part[kAttnWarps];
    __shared__ int found_b;
    __shared__ int64_t found_rest;
    __shared__ float warp_m[kAttnWarps][16], warp_l[kAttnWarps][16];
    __shared__ uint32_t stage_mask[kAttnWarps][kAttnStages];
    __shared__ int join_now;

    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, j4 = lane & 3;
    const int HV = p.segments_per_sequence;
    const int B = p.a.batch;
    uint8_t* ring = smem + (size_t)warp * kAttnStages * S::kStageBytes;
    longlong2* addr = reinterpret_cast<longlong2*>(smem + S::kRingBytes) + warp * kAttnWarpTokens;
    float* merge = reinterpret_cast<float*>(smem + S::kRingBytes + S::kAddrBytes);

    auto out_row = [&](int b, int head) { return static_cast<TQ*>(p.a.out) + b * p.a.out_batch + head * p.a.out_head; };

    // ---------------------------------------------------------------- this CTA's range of tiles
    // Sum of all sequences' tiles, and empty sequences' outputs on the way.
    int64_t mine = 0;
    for (int b = threadIdx.x; b < B; b += kAttnThreads) {
        int first, length;
        sequence_span(p, b, first, length);
        mine += (int64_t)tiles_of(first, length) * HV;
    }
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) scan_part[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) total += scan_part[w];
    if (total == 0) return;
    // Small problems leave CTAs idle rather than cut segments below kAttnMinTiles tiles a CTA.
    const int ctas = (int)min((int64_t)gridDim.x, (total + kAttnMinTiles - 1) / kAttnMinTiles);
    if ((int)blockIdx.x >= ctas) return;
    const int64_t range0 = total * blockIdx.x / ctas, range1 = total * (blockIdx.x + 1) / ctas;
    // The sequence that holds tile range0: scan 128 sequences at a time.
    int64_t before = 0;
    for (int base = 0; base < B; base += kAttnThreads) {
        const int b = base + threadIdx.x;
        int64_t v = 0;
        if (b < B) {
            int first, length;
            sequence_span(p, b, first, length);
            v = (int64_t)tiles_of(first, length) * HV;
        }
        int64_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();
        if (lane == 31) scan_part[warp] = incl;
        __syncthreads();
        int64_t lo = before + incl - v;
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            if (w < warp) lo += scan_part[w];
            all += scan_part[w];
        }
        if (range0 >= lo && range0 < lo + v) {
            found_b = b;
            found_rest = range0 - lo;
        }
        before += all;
        if (before > range0) break;
    }
    __syncthreads();
    const int steps = (int)(range1 - range0);

    TileWalk at;      // the step being computed
    at.b = found_b;
    sequence_span(p, at.b, at.first, at.length);
    at.tiles = tiles_of(at.first, at.length);
    at.hv = (int)(found_rest / at.tiles);
    at.tile = (int)(found_rest - (int64_t)at.hv * at.tiles);
    TileWalk ahead = at;   // the step whose addresses are fetched next
    auto advance = [&](TileWalk& w) {
        if (++w.tile < w.tiles) return;
        w.tile = 0;
        if (++w.hv < HV) return;
        w.hv = 0;
        do {
            if (++w.b >= B) return;      // past the last tile: not used
            sequence_span(p, w.b, w.first, w.length);
            w.tiles = tiles_of(w.first, w.length);
        } while (w.tiles == 0);
    };

    // ---------------------------------------------------------------- copies
    // Lane r < 16 fetches the page of its row r of the next step; the number is used one step later.
    int next_page = -1, next_place = 0, next_head = 0;
    auto fetch = [&]() {
        const int64_t pos = (int64_t)ahead.first + (int64_t)ahead.tile * kAttnTile + warp * kAttnWarpTokens + (lane & 15);
        next_page = -1;
        next_head = ahead.hv / p.head_groups;
        if (pos < ahead.length) {
            const int col = p.page_shift >= 0 ? (int)pos >> p.page_shift : (int)pos / p.page_size;
            next_place = (int)pos - col * p.page_size;
            next_page = p.a.block_table[ahead.b * p.a.table_stride + col];
        }
        advance(ahead);
    };
    const uint8_t* kbase = static_cast<const uint8_t*>(p.a.k_cache);
    const uint8_t* vbase = static_cast<const uint8_t*>(p.a.v_cache);
    const int row_chunks = p.head_dim * (FP8 ? 1 : 2) / 16;
    auto issue = [&](int stage) {
        const bool have = lane < 16 && next_page >= 0 && next_page < p.a.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, have);
        if (lane < 16) {
            const int64_t pg = have ? next_page : 0, pl = have ? next_place : 0;
            longlong2 o;
            o.x = (pg * p.a.k_page + pl * p.a.k_place + next_head * p.a.k_head) * (FP8 ? 1 : 2);
            o.y = (pg * p.a.v_page + pl * p.a.v_place + next_head * p.a.v_head) * (FP8 ? 1 : 2);
            addr[lane] = o;
        }
        if (lane == 0) stage_mask[warp][stage] = mask;
        __syncwarp();
        if (mask) {
            const uint32_t dst = smem_u32(ring + (size_t)stage * S::kStageBytes);
            constexpr int kAll = kAttnWarpTokens * S::kChunks;
#pragma unroll
            for (int i = 0; i < (kAll + 31) / 32; ++i) {
                const int idx = lane + 32 * i;
                if (kAll % 32 != 0 && idx >= kAll) break;
                const int row = idx / S::kChunks, ch = idx - row * S::kChunks;
                const longlong2 o = addr[row];
                const bool in = ((mask >> row) & 1u) && ch < row_chunks;
                const uint32_t d = dst + row * S::kPitch + ch * 16;
                cp_async_16_zfill(d, in ? kbase + o.x + ch * 16 : kbase, in ? 16u : 0u);
                cp_async_16_zfill(d + S::kRowsBytes, in ? vbase + o.y + ch * 16 : vbase, in ? 16u : 0u);
            }
        }
        cp_async_commit();
        __syncwarp();
    };

    // ---------------------------------------------------------------- state of the running softmax
    uint32_t q[KD][4];
    float o[2 * KD][4];
    float m0 = -FLT_MAX, m1 = -FLT_MAX, l0 = 0.f, l1 = 0.f;   // rows quad and quad + 8
    float sc0 = 0.f, sc1 = 0.f;                               // score -> log2 units
    int rows = 0, head0 = 0;
    bool first_segment = true;

    auto load_query = [&]() {
        const int kvh = at.hv / p.head_groups, hg = at.hv - kvh * p.head_groups;
        head0 = kvh * p.group + hg * 16;
        rows = min(16, p.group - hg * 16);
        const TQ* q0 = static_cast<const TQ*>(p.a.q) + at.b * p.a.q_batch + (int64_t)(head0 + quad) * p.a.q_head;
        const TQ* q1 = q0 + 8 * p.a.q_head;
        const bool in0 = quad < rows, in1 = quad + 8 < rows;
#pragma unroll
        for (int kk = 0; kk < KD; ++kk) {
            // the two element pairs of this lane: (2j, 2j+1) and (2j+8, 2j+9), or, for E4M3 caches, four neighbours
            // (the product's order over the head dimension is free; see the key fragments)
            const int da = kk * 16 + (FP8 ? 4 * j4 : 2 * j4), db = FP8 ? da + 2 : da + 8;
            q[kk][0] = in0 && da < p.head_dim ? *reinterpret_cast<const uint32_t*>(q0 + da) : 0u;
            q[kk][1] = in1 && da < p.head_dim ? *reinterpret_cast<const uint32_t*>(q1 + da) : 0u;
            q[kk][2] = in0 && db < p.head_dim ? *reinterpret_cast<const uint32_t*>(q0 + db) : 0u;
            q[kk][3] = in1 && db < p.head_dim ? *reinterpret_cast<const uint32_t*>(q1 + db) : 0u;
        }
        sc0 = sc1 = p.score_log2;
        if constexpr (FP8 && !std::is_same<T, TQ>::value) {
            // bf16 queries against f16 keys: each row is scaled by a power of two to a largest element in [1, 2)
            // (exact; elements 2^-24 of the largest and smaller lose bits) and its scores are scaled back
            float top0 = 0.f, top1 = 0.f;
#pragma unroll
            for (int kk = 0; kk < KD; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = unpack2<TQ>(q[kk][i]);
                    float& top = (i & 1) ? top1 : top0;
                    top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                }
#pragma unroll
            for (int s = 1; s < 4; s <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, s));
                top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, s));
            }
            // biased exponents, kept where 2^e and 2^-e are normal numbers
            const int e0 = min(max((int)(__float_as_uint(top0) >> 23), 1), 252);
            const int e1 = min(max((int)(__float_as_uint(top1) >> 23), 1), 252);
            const float d0 = __uint_as_float((uint32_t)(254 - e0) << 23), d1 = __uint_as_float((uint32_t)(254 - e1) << 23);
            sc0 *= __uint_as_float((uint32_t)e0 << 23);
            sc1 *= __uint_as_float((uint32_t)e1 << 23);
#pragma unroll
            for (int kk = 0; kk < KD; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = unpack2<TQ>(q[kk][i]);
                    const float d = (i & 1) ? d1 : d0;
                    q[kk][i] = round2<T>(v.x * d, v.y * d);
                }
        }
#pragma unroll
        for (int n = 0; n < 2 * KD; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        m0 = m1 = -FLT_MAX;
        l0 = l1 = 0.f;
    };

    auto compute = [&](int stage) {
        const uint32_t mask = stage_mask[warp][stage];
        if (!mask) return;
        const uint32_t ks = smem_u32(ring + (size_t)stage * S::kStageBytes), vs = ks + S::kRowsBytes;
        float s[2][4] = {};
        if constexpr (FP8) {
            // one 32-bit word of a lane is four neighbouring elements of its row: two f16 pairs, the b0 and b1 of one step
            const uint32_t row = (lane & 7) + ((lane >> 3) & 1) * 8;
            const uint32_t base = ks + row * S::kPitch + (lane >> 4) * 16;
#pragma unroll
            for (int kk = 0; kk < KD; kk += 2) {
                if (kk + 1 < KD) {
                    uint32_t r[4];
                    ldmatrix_x4(base + kk * 16, r);
                    mma_16816<T>(s[0], q[kk], e4m3x2_to_half2(r[0]), e4m3x2_to_half2(r[0] >> 16));
                    mma_16816<T>(s[1], q[kk], e4m3x2_to_half2(r[1]), e4m3x2_to_half2(r[1] >> 16));
                    mma_16816<T>(s[0], q[kk + 1], e4m3x2_to_half2(r[2]), e4m3x2_to_half2(r[2] >> 16));
                    mma_16816<T>(s[1], q[kk + 1], e4m3x2_to_half2(r[3]), e4m3x2_to_half2(r[3] >> 16));
                } else {
                    uint32_t r[2];
                    ldmatrix_x2(ks + (lane & 15) * S::kPitch + kk * 16, r);
                    mma_16816<T>(s[0], q[kk], e4m3x2_to_half2(r[0]), e4m3x2_to_half2(r[0] >> 16));
                    mma_16816<T>(s[1], q[kk], e4m3x2_to_half2(r[1]), e4m3x2_to_half2(r[1] >> 16));
                }
            }
        } else {
            const uint32_t row = (lane & 7) + (lane >> 4) * 8;
            const uint32_t base = ks + row * S::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int kk = 0; kk < KD; ++kk) {
                uint32_t r[4];
                ldmatrix_x4(base + kk * 32, r);
                mma_16816<T>(s[0], q[kk], r[0], r[1]);
                mma_16816<T>(s[1], q[kk], r[2], r[3]);
            }
        }
        // scores in log2 units; masked positions to -inf
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[n][0] *= sc0;
            s[n][1] *= sc0;
            s[n][2] *= sc1;
            s[n][3] *= sc1;
        }
        if (mask != 0xFFFFu) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!((mask >> (n * 8 + 2 * j4 + i)) & 1u)) s[n][i] = s[n][i + 2] = -INFINITY;
        }
        float top0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float top1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, d));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, d));
        }
        if (__any_sync(0xffffffffu, top0 > m0 || top1 > m1)) {
            const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
            const float f0 = exp2_fast(m0 - n0), f1 = exp2_fast(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int n = 0; n < 2 * KD; ++n) {
                o[n][0] *= f0;
                o[n][1] *= f0;
                o[n][2] *= f1;
                o[n][3] *= f1;
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[n][0] = exp2_fast(s[n][0] - m0);
            s[n][1] = exp2_fast(s[n][1] - m0);
            s[n][2] = exp2_fast(s[n][2] - m1);
            s[n][3] = exp2_fast(s[n][3] - m1);
            l0 += s[n][0] + s[n][1];
            l1 += s[n][2] + s[n][3];
        }
        // Probabilities as the 16-bit left operand of the product with V (the matrix instruction takes 16-bit operands);
        // their sum l is taken in fp32 before that rounding, O stays fp32.
        const uint32_t a[4] = {round2<T>(s[0][0], s[0][1]), round2<T>(s[0][2], s[0][3]),
                               round2<T>(s[1][0], s[1][1]), round2<T>(s[1][2], s[1][3])};
        const uint32_t vrow = vs + ((lane & 7) + ((lane >> 3) & 1) * 8) * S::kPitch;
        if constexpr (FP8) {
            // a transposed load moves pairs of elements: bytes (t0 d0, t0 d1, t1 d0, t1 d1); reordered to pairs of
            // tokens, the even elements of a 16-element block form one 8-column tile and the odd ones another
            auto tile = [&](int blk, uint32_t lo, uint32_t hi) {
                const uint32_t x = __byte_perm(lo, 0u, 0x3120), y = __byte_perm(hi, 0u, 0x3120);
                mma_16816<T>(o[2 * blk], a, e4m3x2_to_half2(x), e4m3x2_to_half2(y));
                mma_16816<T>(o[2 * blk + 1], a, e4m3x2_to_half2(x >> 16), e4m3x2_to_half2(y >> 16));
            };
#pragma unroll
            for (int blk = 0; blk < KD; blk += 2) {
                uint32_t r[4];
                // the last odd block loads its own chunk twice
                ldmatrix_x4_trans(vrow + (blk + (blk + 1 < KD ? (lane >> 4) : 0)) * 16, r);
                tile(blk, r[0], r[1]);
                if (blk + 1 < KD) tile(blk + 1, r[2], r[3]);
            }
        } else {
#pragma unroll
            for (int blk = 0; blk < KD; ++blk) {
                uint32_t r[4];
                ldmatrix_x4_trans(vrow + blk * 32 + (lane >> 4) * 16, r);
                mma_16816<T>(o[2 * blk], a, r[0], r[1]);
                mma_16816<T>(o[2 * blk + 1], a, r[2], r[3]);
            }
        }
    };

    // This thread's elements of O as (row, column) pairs: fn(row, dim, value).
    auto each_o = [&](auto&& fn) {
#pragma unroll
        for (int blk = 0; blk < KD; ++blk)
#pragma unroll
            for (int h = 0; h < 2; ++h) {        // rows quad, quad + 8
                const int r = quad + 8 * h;
                if constexpr (FP8) {
                    const int d = blk * 16 + 4 * j4;
                    fn(r, d, o[2 * blk][2 * h], o[2 * blk + 1][2 * h]);
                    fn(r, d + 2, o[2 * blk][2 * h + 1], o[2 * blk + 1][2 * h + 1]);
                } else {
                    const int d = blk * 16 + 2 * j4;
                    fn(r, d, o[2 * blk][2 * h], o[2 * blk][2 * h + 1]);
                    fn(r, d + 8, o[2 * blk + 1][2 * h], o[2 * blk + 1][2 * h + 1]);
                }
            }
    };
    constexpr float kLn2 = 0.693147180559945309f;
    auto write_lse = [&](int b, int row, float m, float l) {
        if (p.a.lse) p.a.lse[(int64_t)b * p.heads + head0 + row] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
    };

    // The segment's positions of this CTA are done: join the warps, then write or leave a partial.
    auto flush = [&](int64_t tile_index) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        if (j4 == 0) {
            warp_m[warp][quad] = m0;
            warp_m[warp][quad + 8] = m1;
            warp_l[warp][quad] = l0;
            warp_l[warp][quad + 8] = l1;
        }
        __syncthreads();
        float M0 = -FLT_MAX, M1 = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            M0 = fmaxf(M0, warp_m[w][quad]);
            M1 = fmaxf(M1, warp_m[w][quad + 8]);
        }
        const float f0 = exp2_fast(m0 - M0), f1 = exp2_fast(m1 - M1);
        // one warp after the other adds its share (a fixed order)
        for (int w = 0; w < kAttnWarps; ++w) {
            if (warp == w)
                each_o([&](int r, int d, float x, float y) {
                    if (r >= rows) return;
                    const float f = r < 8 ? f0 : f1;
                    float2* at2 = reinterpret_cast<float2*>(merge + r * S::kMergePitch + d);
                    float2 v = make_float2(x * f, y * f);
                    if (w > 0) {
                        v.x += at2->x;
                        v.y += at2->y;
                    }
                    *at2 = v;
                });
            __syncthreads();
        }
        auto row_ml = [&](int r, float& m, float& l) {
            m = -FLT_MAX;
            l = 0.f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, warp_m[w][r]);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) l = fmaf(warp_l[w][r], exp2_fast(warp_m[w][r] - m), l);
        };
        const int64_t seg0 = tile_index - at.tile, seg1 = seg0 + at.tiles;   // the segment's tiles
        const int quarter = p.head_dim / 4;
        if (seg0 >= range0 && seg1 <= range1) {
            for (int i = threadIdx.x; i < rows * quarter; i += kAttnThreads) {
                const int r = i / quarter, d = (i - r * quarter) * 4;
                float m, l;
                row_ml(r, m, l);
                const float4 v = *reinterpret_cast<const float4*>(merge + r * S::kMergePitch + d);
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
            __stcg(reinterpret_cast<float4*>(slot + r * S::kDim + d), *reinterpret_cast<const float4*>(merge + r * S::kMergePitch + d));
        }
        if (threadIdx.x < rows) {
            float m, l;
            row_ml(threadIdx.x, m, l);
            __stcg(slot + 16 * S::kDim + threadIdx.x, m);
            __stcg(slot + 16 * S::kDim + 16 + threadIdx.x, l);
        }
        // the CTAs that share the segment: those of its first and last tile and all between
        const int c0 = (int)(((seg0 + 1) * ctas - 1) / total), c1 = (int)((seg1 * ctas - 1) / total);
        uint32_t* counter = p.counters + (int64_t)at.b * HV + at.hv;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) join_now = atomicAdd(counter, 1u) == (uint32_t)(c1 - c0);
        __syncthreads();
        if (join_now) {
            __threadfence();
            const bool c0_first = total * c0 / ctas == seg0;
            auto slot_of = [&](int c) {
                return p.partials + ((int64_t)c * 2 + (c == c0 && !c0_first ? 1 : 0)) * S::kSlotFloats;
            };
            for (int i = threadIdx.x; i < rows * quarter; i += kAttnThreads) {
                const int r = i / quarter, d = (i - r * quarter) * 4;
                float M = -FLT_MAX, L = 0.f;
#pragma unroll 8
                for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(slot_of(c) + 16 * S::kDim + r));
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int c = c0; c <= c1; ++c) {
                    const float* sl = slot_of(c);
                    const float f = exp2_fast(__ldcg(sl + 16 * S::kDim + r) - M);
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(sl + r * S::kDim + d));
                    L = fmaf(__ldcg(sl + 16 * S::kDim + 16 + r), f, L);
                    v.x = fmaf(x.x, f, v.x);
                    v.y = fmaf(x.y, f, v.y);
                    v.z = fmaf(x.z, f, v.z);
                    v.w = fmaf(x.w, f, v.w);
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
    fetch();
#pragma unroll
    for (int i = 0; i < kAttnStages - 1; ++i) {
        if (i < steps) {
            issue(i);
            if (i + 1 < steps) fetch();
        } else {
            cp_async_commit();
        }
    }
    load_query();
    int stage = 0, fill = kAttnStages - 1;
    for (int i = 0; i < steps; ++i) {
        cp_async_wait<kAttnStages - 2>();
        __syncwarp();
        // the slot computed on in the previous step is free
        if (i + kAttnStages - 1 < steps) {
            issue(fill);
            if (i + kAttnStages < steps) fetch();
        } else {
            cp_async_commit();
        }
        compute(stage);
        if (at.tile + 1 == at.tiles || i + 1 == steps) {
            flush(range0 + i);
            first_segment = false;
            if (i + 1 < steps) {
                advance(at);
                load_query();
            }
        } else {
            ++at.tile;
        }
        if (++stage == kAttnStages) stage = 0;
        if (++fill == kAttnStages) fill = 0;
    }
    cp_async_wait<0>();
}

template <typename T, typename TQ, bool FP8, int KD>
cudaError_t attn_launch(const AttnParams& p, int grid, cudaStream_t stream) {
    return launch_dependent(paged_attn_kernel<T, TQ, FP8, KD>, dim3((unsigned)grid), dim3(kAttnThreads), AttnShape<KD, FP8>::kSmemBytes,
                            stream, p);
}

// Raises the kernel's shared-memory limit and says how many CTAs an SM holds.
template <typename T, typename TQ, bool FP8, int KD>
cudaError_t attn_prepare(AttnVariant* v) {
    using S = AttnShape<KD, FP8>;
    auto kern = paged_attn_kernel<T, TQ, FP8, KD>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
    if (e != cudaSuccess) return e;
    v->smem_bytes = S::kSmemBytes;
    v->slot_floats = S::kSlotFloats;
    v->launch = &attn_launch<T, TQ, FP8, KD>;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v->ctas_per_sm, kern, kAttnThreads, S::kSmemBytes);
}

// The head sizes held: head_dim is rounded up to one of them.
template <typename T, typename TQ, bool FP8>
cudaError_t attn_variant(int head_dim, AttnVariant* v) {
    if (head_dim <= 64) return attn_prepare<T, TQ, FP8, 4>(v);
    if (head_dim <= 80) return attn_prepare<T, TQ, FP8, 5>(v);
    if (head_dim <= 96) return attn_prepare<T, TQ, FP8, 6>(v);
    if (head_dim <= 128) return attn_prepare<T, TQ, FP8, 8>(v);
    return attn_prepare<T, TQ, FP8, 16>(v);
}

}  // namespace dgb
