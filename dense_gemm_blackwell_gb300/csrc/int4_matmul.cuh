// int4_matmul.cuh -- Y = X W^T for up to 16 tokens, W in 4-bit codes with group
// scales, alone or as a gated pair (include/feedforward.h): one stream over W.
//
// A warp multiplies 16 rows of W (of a gated pair: 8 gates and the 8 columns they
// multiply) by 8 or 16 tokens with 16 x 8 x 16 matrix instructions, W on the 16-row
// side, straight from global memory: which 16 of K's elements one instruction takes is
// free as long as both operands agree, so each lane loads consecutive ones of its two
// rows, 16 of every 64 bytes (four lanes exchange words where groups are shorter than
// what they load together), and no weight passes through shared memory.  X lies there, laid out once per block so that a lane's part of an
// instruction pair is one 16-byte load.  A block's warps share a tile's K (several
// tiles where K is short); a block goes from tile to tile with the next stage's weights
// on the way, across tiles too, and two blocks an SM cover each other's joins.  The CTAs
// of a cluster share K when there are few tiles or X does not fit.  All sums are fp32 in
// a fixed order, so a column's sum never depends on timing.
//
// A code is a 16-bit float as it stands: the integers 0..255 in the low bits of an f16 are
// the multiples of its least step 2^-24, of a bf16 those of 2^-133 (subnormal numbers and
// the binade above them, which matrix instructions take exactly).  So four pairs of codes of
// a word need one bitwise operation each and one shift: bits 0..3 of each half are code *
// step, bits 4..7 code * 16 step; their x is divided by 16 in advance (bf16) or their sums
// are.  (Adding a code to the bits of a float 2^7 and subtracting 2^7 + z takes 11
// instructions for eight codes, this 5; bitwise operations run at half rate.)  Tokens in
// bf16 are multiplied by 2^64, so that products stay far from fp32's subnormal numbers.  Zero
// points come in as z times the sum of X over the group's part of a chunk:
// s (sum q x - z sum x), every factor and sum in fp32, nothing rounded to 16 bits.
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "activation.cuh"
#include "common.cuh"
#include "elem.cuh"
#include "int4_matmul.h"

namespace dgb {

constexpr int kInt4Threads = 32 * kInt4Warps;
constexpr int kInt4Pitch = 17;           // floats between tokens of a warp's sums: 16 rows

// What the sums of code * x are multiplied by when they are complete, its reciprocal, and x as the instructions take it.
template <typename T>
struct CodeScale;
template <>
struct CodeScale<__nv_bfloat16> {
    static constexpr float back = 0x1p69f, step = 0x1p-69f;         // 2^(133 - 64)
    static constexpr bool even_out = true;      // x of codes in bits 4..7 is divided by 16, exactly
    static __device__ __forceinline__ uint32_t operand(uint32_t x, bool high) {
        uint32_t r;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(high ? 0x5D805D80u : 0x5F805F80u));      // 2^60 or 2^64
        return r;
    }
};
template <>
struct CodeScale<__half> {
    static constexpr float back = 0x1p24f, step = 0x1p-24f;
    static constexpr bool even_out = false;     // it might lose bits of a small one: the sums are told apart, or the codes shifted
    static __device__ __forceinline__ uint32_t operand(uint32_t x, bool) { return x; }
};

// `bytes` (may be over 16 or negative) bytes of p's 16, the rest as zeros; elements of 2 bytes.  Not by the read-only path: the
// kernel before this one, which may still run when this one starts, may have written them.
__device__ __forceinline__ uint4 load_clipped16(const void* p, int bytes) {
    if (bytes >= 16) return *static_cast<const uint4*>(p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (2 * i + 2 <= bytes) w[i >> 1] |= (uint32_t)static_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same byte by byte.
__device__ __forceinline__ uint4 load_clipped_bytes(const void* p, int bytes) {
    if (bytes >= 16) return __ldg(static_cast<const uint4*>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (bytes > 0) {
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (i < bytes) w[i >> 2] |= (uint32_t)__ldg(static_cast<const uint8_t*>(p) + i) << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// weights: read once by the whole grid
__device__ __forceinline__ uint4 load_once16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// 16 words of a row, lane t of four holding 4 t .. 4 t + 3, dealt out so that the lanes share every chunk of 4 VEC words: w[c VEC + v]
// becomes a word of chunk c, of VEC = 1 (a transposition) word t, of VEC = 2 words 2 rank + v with the lane's rank below.
template <int VEC>
__device__ __forceinline__ void deal_words(uint32_t (&w)[4], int t) {
    if constexpr (VEC <= 2) {
        const bool up = (t & 2) != 0;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[2], 2), b = __shfl_xor_sync(0xffffffffu, up ? w[1] : w[3], 2);
        if (up) {
            w[0] = a;
            w[1] = b;
        } else {
            w[2] = a;
            w[3] = b;
        }
    }
    if constexpr (VEC == 1) {
        const bool odd = (t & 1) != 0;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
        if (odd) {
            w[0] = a;
            w[2] = b;
        } else {
            w[1] = a;
            w[3] = b;
        }
    }
}

// A lane's place among the four of a chunk.
template <int VEC>
__device__ __forceinline__ int chunk_rank(int t) { return VEC == 2 ? (t & 1) * 2 + (t >> 1) : t; }

// VEC: consecutive 32-bit words of a row (eight codes each) that a lane takes: four lanes' make a chunk, which lies in one group.
template <typename T, int VEC, int NB, bool GATED>
__global__ void __launch_bounds__(kInt4Threads, 2) int4_matmul_kernel(const __grid_constant__ Int4Params p) {
    constexpr int kRowWords = kInt4RowBytes / 16;            // of a stage and lane
    constexpr int kChunks = kRowWords / VEC, kChunkK = 32 * VEC, kStageK = kChunks * kChunkK;
    constexpr int kTokens = 8 * NB;
    constexpr int kFactors = VEC == 1 ? 4 : VEC == 2 ? 2 : 1;       // groups of a stage: 4 of these at most
    constexpr int kOut = GATED ? 8 : 16;                    // columns of Y of a tile

    extern __shared__ uint4 int4_smem[];
    float* sums = reinterpret_cast<float*>(int4_smem);       // [2][warp][token][kInt4Pitch]
    // [warp][group of the stage][row]: scale and zero point
    float2* factors = reinterpret_cast<float2*>(sums + 2 * kInt4Warps * kTokens * kInt4Pitch) + (threadIdx.x >> 5) * (4 * kFactors * 16);
    float* x_sums = sums + 2 * kInt4Warps * kTokens * kInt4Pitch + kInt4Warps * 4 * kFactors * 16 * 2;      // [chunk][token]: sum of X, in steps
    // [stage][word][NB][lane]

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int KS = 1 << p.k_split_log, rank = KS > 1 ? (int)cluster_ctarank() : 0;
    const int KW = 1 << p.k_warps_log, share = warp & (KW - 1), sub = warp >> p.k_warps_log;    // of the warps that share a tile; which of the block's tiles
    const int per_round = kInt4Warps >> p.k_warps_log;                   // tiles of a block at a time
    const int clusters = (int)gridDim.x >> p.k_split_log, cluster = (int)blockIdx.x >> p.k_split_log;

    const int stages = (p.k + kStageK - 1) / kStageK, whole = p.k / kStageK;
    const int s0 = (int)(((int64_t)stages * rank) >> p.k_split_log), s_count = (int)(((int64_t)stages * (rank + 1)) >> p.k_split_log) - s0;
    const int per_tile = (s_count + KW - 1) >> p.k_warps_log;           // stages of a warp in a tile
    const int own = s_count > share ? (s_count - share + KW - 1) >> p.k_warps_log : 0;     // of which this one has so many, the rest lie past the end
    const int tiles = (p.n + kOut - 1) / kOut;
    const int rounds = p.rounds;
    uint4* x_smem = reinterpret_cast<uint4*>(x_sums + s_count * kChunks * kTokens);
    // The warp's tile in round r; there may be none.  Its stages in this CTA's part of K: share, share + KW, ...
    auto tile_of = [&](int r) { return (r * clusters + cluster) * per_round + sub; };
    // Row g + 8 i of a tile; rows past the last are that one again and are not stored.
    auto row_of = [&](int tile, int i) {
        return GATED ? (int64_t)i * p.n + min(tile * kOut + g, p.n - 1) : (int64_t)min(tile * kOut + 8 * i + g, p.n - 1);
    };
    // ---------------------------------------------------------------- weights, a stage ahead in registers
    int load_round = 0, load_at = 0;
    bool load_tile = false;
    const uint8_t* from[2];
    auto set_rows = [&] {
        const int tile = tile_of(load_round);
        load_tile = load_round < rounds && tile < tiles;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            from[i] = static_cast<const uint8_t*>(p.w) + row_of(tile, i) * p.ldw_bytes + (int64_t)(s0 + share) * kInt4RowBytes + 16 * t;
    };
    // The lines of the stage that is loaded next into L2, four lanes a row pair's four lines: its loads are issued a stage later and
    // used a stage after that, which alone does not cover DRAM's latency under load.
    auto prefetch = [&] {
        if (load_tile && load_at < own && s0 + share + (load_at << p.k_warps_log) < whole)
            asm volatile("prefetch.global.L2 [%0];" ::"l"((t & 1 ? from[1] : from[0]) + (128 * (t >> 1) - 16 * t)));
    };
    auto load = [&](uint4 (&w)[2][kRowWords / 4]) {       // 16 bytes of every 64 of a row
        if (load_tile && load_at < own) {
            const int stage = s0 + share + (load_at << p.k_warps_log);
            if (stage < whole) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < kRowWords / 4; ++s) w[i][s] = load_once16(from[i] + 64 * s);
            } else {
                const int left = p.k / 2 - stage * kInt4RowBytes - 16 * t;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < kRowWords / 4; ++s) w[i][s] = load_clipped_bytes(from[i] + 64 * s, left - 64 * s);
            }
        }
        if (++load_at < per_tile) {
#pragma unroll
            for (int i = 0; i < 2; ++i) from[i] += KW * kInt4RowBytes;
        } else {
            load_at = 0;
            ++load_round;
            set_rows();
        }
        prefetch();
    };
    // ---------------------------------------------------------------- scales and zero points, a stage ahead in registers
    // A lane of row g (and g + 8) has the stage's groups t, t + 4, ...; they stay as loaded until the stage comes, as whatever uses
    // them would wait for them.
    int look_round = 0, look_at = 0;
    bool look_tile = false;
    uint16_t scale_next[2][kFactors] = {};
    uint8_t zero_next[2][kFactors] = {};
    int in_group_next = 0;      // where in its group the stage begins, in 32s
    const uint16_t* scale_row[2];
    const uint8_t* zero_row[2];
    const int last_group = (p.k - 1) / p.group, group_units = p.group / 32;
    auto set_looks = [&] {
        const int tile = tile_of(look_round);
        look_tile = look_round < rounds && tile < tiles;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = row_of(tile, i);
            scale_row[i] = static_cast<const uint16_t*>(p.scales) + row * p.ld_scales;
            zero_row[i] = p.zeros + (p.zeros ? row * p.ld_zeros : 0);
        }
    };
    auto look = [&] {
        if (look_tile && look_at < own) {
            const uint32_t unit = (uint32_t)(s0 + share + (look_at << p.k_warps_log)) * (kStageK / 32);
            int first = (int)__umulhi(unit, p.group_magic);
            in_group_next = (int)unit - first * group_units;
            if (in_group_next >= group_units) {
                in_group_next -= group_units;
                ++first;
            }
#pragma unroll
            for (int h = 0; h < kFactors; ++h) {
                const int gi = min(first + t + 4 * h, last_group);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    scale_next[i][h] = __ldg(scale_row[i] + gi);
                    zero_next[i][h] = p.zeros ? __ldg(zero_row[i] + gi) : (uint8_t)8;
                }
            }
        }
        if (++look_at == per_tile) {
            look_at = 0;
            ++look_round;
            set_looks();
        }
    };

    uint4 next[2][kRowWords / 4];
    uint32_t now[2][kRowWords];
    set_rows();
    prefetch();         // while the kernel before this one may still run: it returns nothing, so it does not matter who writes W
    griddep_wait();
    griddep_launch_dependents();
    load(next);
    set_looks();
    look();
    // X of this CTA's part of K and its sums over the chunks, a quarter of a token's chunk at a time; zeros past K.  What lies in the
    // places of tokens past the last is never stored: a column of the products depends on its own token alone.
    {
        constexpr int kBatch = 8 / VEC;         // quarters whose loads are on the way
        const int chunks = s_count * kChunks, quarters = (chunks * 4) << p.tokens_log;
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + s0 * kStageK;
        const int k_left = p.k - s0 * kStageK;
        for (int all0 = 0; all0 < quarters; all0 += kBatch * kInt4Threads) {       // the same turns in every lane: they exchange sums
            const int e0 = all0 + (int)threadIdx.x;
            uint4 q[kBatch][VEC];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int e = e0 + b * kInt4Threads, m = (e >> 2) & ((1 << p.tokens_log) - 1), c = e >> (2 + p.tokens_log);
                const bool there = e < quarters && m < p.tokens;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const int k = c * kChunkK + (chunk_rank<VEC>(t) * VEC + v) * 8;
                    q[b][v] = make_uint4(0u, 0u, 0u, 0u);
                    if (there && k < k_left) q[b][v] = load_clipped16(x + (int64_t)m * p.ldx + k, 2 * (k_left - k));
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int e = e0 + b * kInt4Threads, m = (e >> 2) & ((1 << p.tokens_log) - 1), c = e >> (2 + p.tokens_log);
                if (all0 + b * kInt4Threads >= quarters) break;
                float sum = 0.f;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float f[8];
                    unpack8<T>(q[b][v], f);
                    sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
                    // elements j and j + 4 of a word of codes lie 16 bits apart: 0 and 4, 2 and 6, then 1 and 5, 3 and 7
                    const uint4 o = q[b][v];
                    if (e < quarters && m < p.tokens)
                        x_smem[((c * VEC + v) * NB + (m >> 3)) * 32 + (m & 7) * 4 + t] =
                            make_uint4(CodeScale<T>::operand(__byte_perm(o.x, o.z, 0x5410), false), CodeScale<T>::operand(__byte_perm(o.y, o.w, 0x5410), false),
                                       CodeScale<T>::operand(__byte_perm(o.x, o.z, 0x7632), true), CodeScale<T>::operand(__byte_perm(o.y, o.w, 0x7632), true));
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t == 0 && e < quarters && m < p.tokens) x_sums[c * kTokens + m] = sum * CodeScale<T>::step;
            }
        }
    }
    __syncthreads();

    float acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
    int r = 0, at = 0;
    bool tile_here = tile_of(0) < tiles;
    const int all_stages = rounds * per_tile;
    for (int f = 0; f < all_stages; ++f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < kRowWords / 4; ++s) {
                uint32_t w[4] = {next[i][s].x, next[i][s].y, next[i][s].z, next[i][s].w};
                deal_words<VEC>(w, t);
#pragma unroll
                for (int j = 0; j < 4; ++j) now[i][4 * s + j] = w[j];
            }
        load(next);
        __syncwarp();           // every lane is done with the stage before
#pragma unroll
        for (int h = 0; h < kFactors; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                factors[(t + 4 * h) * 16 + 8 * i + g] = make_float2(unpack2<T>(scale_next[i][h]).x, (float)zero_next[i][h]);
        __syncwarp();
        int in_group = in_group_next;
        look();
        if (tile_here && at < own) {
            const int in = share + (at << p.k_warps_log);
            const uint4* x = x_smem + (size_t)in * (kRowWords * NB * 32) + lane;
            const float* sx = x_sums + in * (kChunks * kTokens) + 2 * t;
            const int chunks = (p.k - (s0 + in) * kStageK + kChunkK - 1) / kChunkK;     // that K reaches
            int gi = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (c >= chunks) break;
                // Sums of code * x in steps.  Two accumulators for 8 tokens, as an accumulator's instructions wait for one another; one for
                // 16, whose two columns of instructions take turns.
                constexpr int kSums = NB == 1 ? 2 : 1;
                constexpr bool kShift = NB > 1 && !CodeScale<T>::even_out;       // codes of bits 4..7 brought to bits 0..3
                float part[kSums][NB][4];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const uint32_t w0 = now[0][c * VEC + v], w1 = now[1][c * VEC + v];
                    const uint32_t low[4] = {w0 & 0x000F000Fu, w1 & 0x000F000Fu, (w0 >> 8) & 0x000F000Fu, (w1 >> 8) & 0x000F000Fu};
                    constexpr uint32_t kHigh = kShift ? 0x000F000Fu : 0x00F000F0u;
                    constexpr int kBy = kShift ? 4 : 0;
                    const uint32_t high[4] = {(w0 >> kBy) & kHigh, (w1 >> kBy) & kHigh, (w0 >> (8 + kBy)) & kHigh, (w1 >> (8 + kBy)) & kHigh};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint4 q = x[((c * VEC + v) * NB + nb) * 32];
                        if (v == 0) mma_16816_fresh<T>(part[0][nb], low, q.x, q.y);
                        else mma_16816<T>(part[0][nb], low, q.x, q.y);
                        if (v == 0 && kSums > 1) mma_16816_fresh<T>(part[kSums - 1][nb], high, q.z, q.w);
                        else mma_16816<T>(part[kSums - 1][nb], high, q.z, q.w);
                    }
                }
                const float2 f0 = factors[gi * 16 + g], f1 = factors[gi * 16 + 8 + g];       // of rows g and g + 8
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float2 s = *reinterpret_cast<const float2*>(sx + c * kTokens + nb * 8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float sum = part[0][nb][i];
                        if constexpr (kSums > 1) sum = CodeScale<T>::even_out ? sum + part[kSums - 1][nb][i] : fmaf(part[kSums - 1][nb][i], 0.0625f, sum);
                        acc[nb][i] = fmaf(i < 2 ? f0.x : f1.x, fmaf(i < 2 ? -f0.y : -f1.y, i & 1 ? s.y : s.x, sum), acc[nb][i]);
                    }
                }
                in_group += kChunkK / 32;
                if (in_group >= group_units) {
                    in_group -= group_units;
                    ++gi;
                }
            }
        }
        if (++at < per_tile) continue;
        at = 0;

        // ------------------------------------------------------------ a tile's end: the warps' sums, then the cluster's, then Y
        float* mine = sums + (r & 1) * (kInt4Warps * kTokens * kInt4Pitch);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mine[(warp * kTokens + nb * 8 + 2 * t + (i & 1)) * kInt4Pitch + (i >> 1) * 8 + g] = acc[nb][i];
                acc[nb][i] = 0.f;
            }
        // the tile's warps meet; a buffer is written again two rounds on, after all have met once more
        const int threads = 32 * KW, thread = share * 32 + lane;
        if (KW == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(threads) : "memory");
        float* tile_sums = mine + sub * KW * kTokens * kInt4Pitch;
        auto add_warps = [&](int m, int c) {
            float v = tile_sums[m * kInt4Pitch + c];
#pragma unroll 4
            for (int w = 1; w < KW; ++w) v += tile_sums[(w * kTokens + m) * kInt4Pitch + c];
            return v;
        };
        int m0 = 0, m1 = p.tokens;
        if (KS > 1) {
            // in the place of the first warp's sums; each is read and written by one thread
            for (int e = thread; e < p.tokens * 16; e += threads) tile_sums[e / 16 * kInt4Pitch + e % 16] = add_warps(e / 16, e % 16);
            // a CTA that passes has everyone's sums of this round, and everyone has read those of the round before
            cluster_sync();
            m0 = p.tokens * rank >> p.k_split_log;
            m1 = p.tokens * (rank + 1) >> p.k_split_log;
        }
        for (int e0 = m0 * 16; e0 < m1 * 16; e0 += threads) {
            const int e = e0 + thread, m = min(e / 16, m1 - 1), c = e % 16;
            float v = 0.f;
            if (KS == 1) {
                v = add_warps(m, c);
            } else {
                const uint32_t part = smem_u32(tile_sums + m * kInt4Pitch + c);
                for (int o = 0; o < KS; ++o) {
                    float s;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(s) : "r"(map_to_cta(part, (uint32_t)o)));
                    v += s;
                }
            }
            v *= CodeScale<T>::back;
            const int n = tile_of(r) * kOut + c % kOut;
            const bool there = e < m1 * 16 && n < p.n;
            if constexpr (GATED) {
                const float u = __shfl_down_sync(0xffffffffu, v, 8);       // the column's other sum
                if (there && c < 8) static_cast<T*>(p.y)[(int64_t)m * p.ldy + n] = (T)(activate(p.act, v) * u);
            } else if (there) {
                static_cast<T*>(p.y)[(int64_t)m * p.ldy + n] = (T)v;
            }
        }
        ++r;
        tile_here = tile_of(r) < tiles;
    }
    if (KS > 1) cluster_sync_relaxed();     // peers have read this CTA's sums
}

template <typename T, int VEC, int NB, bool GATED>
static cudaError_t launch_int4_as(const Int4Params& p, cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    auto kern = int4_matmul_kernel<T, VEC, NB, GATED>;
    const cudaError_t e = ensure_smem_limit(kern, (size_t)p.smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.grid);
    cfg.blockDim = dim3(kInt4Threads);
    cfg.dynamicSmemBytes = (size_t)p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1u << p.k_split_log;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.k_split_log > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, int VEC>
static cudaError_t launch_int4_vec(const Int4Params& p, bool gated, cudaStream_t stream) {
    if (p.tokens > 8) return gated ? launch_int4_as<T, VEC, 2, true>(p, stream) : launch_int4_as<T, VEC, 2, false>(p, stream);
    return gated ? launch_int4_as<T, VEC, 1, true>(p, stream) : launch_int4_as<T, VEC, 1, false>(p, stream);
}

template <typename T>
static cudaError_t launch_int4(const Int4Params& p, bool gated, cudaStream_t stream) {
    if (p.group % 128 == 0) return launch_int4_vec<T, 4>(p, gated, stream);
    return p.group % 64 == 0 ? launch_int4_vec<T, 2>(p, gated, stream) : launch_int4_vec<T, 1>(p, gated, stream);
}

}  // namespace dgb
