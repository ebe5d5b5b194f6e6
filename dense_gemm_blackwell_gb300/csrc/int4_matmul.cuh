// int4_matmul.cuh -- Y = X W^T for up to 16 tokens, W in 4-bit codes with group
// scales, alone or as a gated pair (include/feedforward.h): one stream over W.
//
// A warp multiplies 16 rows of W (of a gated pair: 8 gates and the 8 columns they
// multiply) by 8 or 16 tokens with 16 x 8 x 16 matrix instructions, W on the 16-row
// side, straight from global memory: which 16 of K's elements one instruction takes is
// free as long as both operands agree, so each lane loads consecutive ones of its two
// rows, 16 of every 64 bytes (four lanes exchange words where groups are shorter than
// what they load together), and no weight passes through shared memory.  X lies there,
// laid out once per block so that a lane's part of an instruction pair is one 16-byte
// load.  (Up to 16 tokens a 128-row tcgen05 tile would be seven eighths empty.)
//
// A block's tiles are laid end to end in stages of 512 codes a row and every warp takes
// an equal run of them, whatever K is: a tile inside a run is stored by its warp, one
// that runs share after the block's only barrier.  (Tiles dealt out whole, or their
// stages in turn, need a barrier a tile: 109 us where runs take 94 at 16 x 4096 x
// 155648.)  The next stage's weights are on the way in registers, across tiles too, and
// the lines of the one after that into L2.  The CTAs of a cluster share K when there are
// few tiles or X does not fit, and join once in a few tiles.  All sums are fp32 in an
// order that the sizes alone decide.
//
// Bound by memory at first and by latency at smaller sizes: a gated pair of 8 tokens, 4096
// -> 2 x 38912 36.9 us (4.5 TB/s; 2 x 77824 64.7 us, 5.2), 2 x 12288 17.1 us (3.1 TB/s:
// 2.2 of a launch, about 3 of bringing X to every block, and 10 or 11 tiles an SM); one
// token 4096 x 4096 4.9 us, of which 1.3 are the bytes.  16 tokens: instructions (195
// TFLOP/s); in groups of 128 these spill 8 to 18 bytes a thread.
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

constexpr int kInt4MaxThreads = 512;
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
__global__ void __launch_bounds__(kInt4MaxThreads, 1) int4_matmul_kernel(const __grid_constant__ Int4Params p) {
    constexpr int kRowWords = kInt4RowBytes / 16;            // of a stage and lane
    constexpr int kChunks = kRowWords / VEC, kChunkK = 32 * VEC, kStageK = kChunks * kChunkK;
    constexpr int kTokens = 8 * NB;
    constexpr int kFactors = VEC == 1 ? 4 : VEC == 2 ? 2 : 1;       // groups of a stage: 4 of these at most
    constexpr int kOut = GATED ? 8 : 16;                    // columns of Y of a tile

    extern __shared__ uint4 int4_smem[];
    __shared__ int tail_tile[kInt4MaxThreads / 32];      // the tile that a warp's run begins and another's ends, or -1
    __shared__ int tile_warps[2][2][kInt4RoundTiles / NB];       // of a cluster's round: the tiles' first and last warps
    const int W = 1 << p.warps_log;
    float* sums = reinterpret_cast<float*>(int4_smem);       // [p.slots][token][kInt4Pitch]
    // [warp][group of the stage][row]: scale and zero point
    float2* factors = reinterpret_cast<float2*>(sums + p.slots * kTokens * kInt4Pitch) + (threadIdx.x >> 5) * (4 * kFactors * 16);
    float* x_sums = sums + p.slots * kTokens * kInt4Pitch + W * 4 * kFactors * 16 * 2;      // [chunk][token]: sum of X, in steps
    // [stage][word][NB][lane]

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int KS = 1 << p.k_split_log, rank = KS > 1 ? (int)cluster_ctarank() : 0;
    const int clusters = (int)gridDim.x >> p.k_split_log, cluster = (int)blockIdx.x >> p.k_split_log;

    const int stages = (p.k + kStageK - 1) / kStageK, whole = p.k / kStageK;
    const int s0 = (int)(((int64_t)stages * rank) >> p.k_split_log), s_count = (int)(((int64_t)stages * (rank + 1)) >> p.k_split_log) - s0;
    const int tiles = (p.n + kOut - 1) / kOut, my_tiles = (tiles - 1 - cluster) / clusters + 1;     // cluster, cluster + clusters, ...
    uint4* x_smem = reinterpret_cast<uint4*>(x_sums + s_count * kChunks * kTokens);
    // Every warp has an equal run of all tiles' stages, tile after tile.  In a cluster: of a round's, up to p.round_tiles tiles with
    // their stages in this CTA's part of K.
    auto tiles_of = [&](int r) { return min(p.round_tiles, my_tiles - r * p.round_tiles); };
    auto units_to = [&](int all, int w) { return all * w >> p.warps_log; };
    // Row g + 8 i of a tile; rows past the last are that one again and are not stored.
    auto row_of = [&](int tile, int i) {
        return GATED ? (int64_t)i * p.n + min(tile * kOut + g, p.n - 1) : (int64_t)min(tile * kOut + 8 * i + g, p.n - 1);
    };
    // ---------------------------------------------------------------- weights, scales and zero points, a stage ahead in registers
    // A lane of row g (and g + 8) has 16 bytes of every 64 of the row's codes and the scales of the stage's groups t, t + 4, ...; they
    // stay as loaded until the stage comes, as whatever uses them would wait for them.
    int a_round = 0, a_left = 0, a_tile = 0, a_stage = 0;       // what is loaded next: a tile of the round and a stage; a_left: 0 = nothing
    const uint8_t* from[2];
    const uint16_t* scale_row[2];
    const uint8_t* zero_row[2];
    uint4 next[2][kRowWords / 4];
    uint16_t scale_next[2][kFactors] = {};
    uint8_t zero_next[2][kFactors] = {};
    int in_group_next = 0;      // where in its group the stage begins, in 32s
    const int last_group = (p.k - 1) / p.group, group_units = p.group / 32;
    auto set_rows = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = row_of((a_round * p.round_tiles + a_tile) * clusters + cluster, i);
            from[i] = static_cast<const uint8_t*>(p.w) + row * p.ldw_bytes + (int64_t)(s0 + a_stage) * kInt4RowBytes + 16 * t;
            scale_row[i] = static_cast<const uint16_t*>(p.scales) + row * p.ld_scales;
            zero_row[i] = p.zeros + (p.zeros ? row * p.ld_zeros : 0);
        }
    };
    auto seek = [&] {       // the warp's first from round a_round on
        for (int count; (count = tiles_of(a_round)) > 0; ++a_round) {
            const int all = count * s_count, u0 = units_to(all, warp);
            if ((a_left = units_to(all, warp + 1) - u0) == 0) continue;
            a_tile = (int)((unsigned)u0 / (unsigned)s_count);
            a_stage = u0 - a_tile * s_count;
            set_rows();
            return;
        }
    };
    // The lines of the stage that is loaded next into L2, four lanes a row pair's four lines: its loads are issued a stage later and
    // used a stage after that, which alone does not cover DRAM's latency under load.
    auto prefetch = [&] {
        if (a_left > 0 && s0 + a_stage < whole)
            asm volatile("prefetch.global.L2 [%0];" ::"l"((t & 1 ? from[1] : from[0]) + (128 * (t >> 1) - 16 * t)));
    };
    auto load_codes = [&] {
        if (a_left == 0) return;
        const int stage = s0 + a_stage;
        if (stage < whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < kRowWords / 4; ++s) next[i][s] = load_once16(from[i] + 64 * s);
        } else {
            const int left = p.k / 2 - stage * kInt4RowBytes - 16 * t;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < kRowWords / 4; ++s) next[i][s] = load_clipped_bytes(from[i] + 64 * s, left - 64 * s);
        }
    };
    auto load_factors = [&] {       // and on to the next stage
        if (a_left == 0) return;
        const uint32_t unit = (uint32_t)(s0 + a_stage) * (kStageK / 32);
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
        if (--a_left == 0) {
            ++a_round;
            seek();
        } else if (++a_stage == s_count) {
            a_stage = 0;
            ++a_tile;
            set_rows();
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) from[i] += kInt4RowBytes;
        }
        prefetch();
    };

    uint32_t now[2][kRowWords];
    seek();
    prefetch();         // while the kernel before this one may still run: it returns nothing, so it does not matter who writes W
    griddep_wait();
    griddep_launch_dependents();
    load_codes();
    load_factors();
    // X of this CTA's part of K and its sums over the chunks, a quarter of a token's chunk at a time; zeros past K.  What lies in the
    // places of tokens past the last is never stored: a column of the products depends on its own token alone.
    {
        constexpr int kBatch = 8 / VEC;         // quarters whose loads are on the way
        const int chunks = s_count * kChunks, quarters = (chunks * 4) << p.tokens_log;
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + s0 * kStageK;
        const int k_left = p.k - s0 * kStageK;
        for (int all0 = 0; all0 < quarters; all0 += kBatch * (int)blockDim.x) {       // the same turns in every lane: they exchange sums
            const int e0 = all0 + (int)threadIdx.x;
            uint4 q[kBatch][VEC];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int e = e0 + b * (int)blockDim.x, m = (e >> 2) & ((1 << p.tokens_log) - 1), c = e >> (2 + p.tokens_log);
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
                const int e = e0 + b * (int)blockDim.x, m = (e >> 2) & ((1 << p.tokens_log) - 1), c = e >> (2 + p.tokens_log);
                if (all0 + b * (int)blockDim.x >= quarters) break;
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

    for (int r = 0, count; (count = tiles_of(r)) > 0; ++r) {
        const int all = count * s_count;
        float* round_sums = sums + (r & 1) * (p.slots / 2 * kTokens * kInt4Pitch);
        int* first_warp = tile_warps[r & 1][0];
        int* last_warp = tile_warps[r & 1][1];
        const int u0 = units_to(all, warp), u1 = units_to(all, warp + 1);
        int tile = (int)((unsigned)u0 / (unsigned)s_count), at = u0 - tile * s_count;      // of the round's tiles; of this CTA's stages
        float acc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
        if (lane == 0) {
            if (KS == 1) tail_tile[warp] = -1;
            else if (at == 0 && u0 < u1) first_warp[tile] = warp;
        }
        bool begun = at == 0;       // this run has the tile's first stage
        for (int u = u0; u < u1; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < kRowWords / 4; ++s) {
                    uint32_t w[4] = {next[i][s].x, next[i][s].y, next[i][s].z, next[i][s].w};
                    deal_words<VEC>(w, t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) now[i][4 * s + j] = w[j];
                }
            load_codes();
            __syncwarp();           // every lane is done with the stage before
#pragma unroll
            for (int h = 0; h < kFactors; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    factors[(t + 4 * h) * 16 + 8 * i + g] = make_float2(unpack2<T>(scale_next[i][h]).x, (float)zero_next[i][h]);
            __syncwarp();
            int in_group = in_group_next;
            load_factors();
            const uint4* x = x_smem + (size_t)at * (kRowWords * NB * 32) + lane;
            const float* sx = x_sums + at * (kChunks * kTokens) + 2 * t;
            const int chunks = (p.k - (s0 + at) * kStageK + kChunkK - 1) / kChunkK;     // that K reaches
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
            if (++at < s_count && u + 1 < u1) continue;
            // the tile's or the run's end
            const bool ended = at == s_count;
            if (KS == 1 && begun && ended) {
                const int n = ((tile * clusters) + cluster) * kOut + g;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int m = nb * 8 + 2 * t + i;
                        const float v0 = acc[nb][i] * CodeScale<T>::back, v1 = acc[nb][2 + i] * CodeScale<T>::back;
                        T* y = static_cast<T*>(p.y) + (int64_t)m * p.ldy + n;
                        if (m < p.tokens && n < p.n) {
                            if constexpr (GATED) *y = (T)(activate(p.act, v0) * v1);
                            else *y = (T)v0;
                        }
                        if (!GATED && m < p.tokens && n + 8 < p.n) y[8] = (T)v1;
                    }
            } else {
                // A run has two parts of tiles at most, of the tile that it does not begin and of the one that it does not end.  In a
                // cluster all sums go this way: from one part to the next either the warp or the tile goes up by one, or both.
                float* mine = round_sums + (KS == 1 ? 2 * warp + begun : warp + tile) * (kTokens * kInt4Pitch);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mine[(nb * 8 + 2 * t + (i & 1)) * kInt4Pitch + (i >> 1) * 8 + g] = acc[nb][i];
                if (lane == 0) {
                    if (KS == 1) {
                        if (begun) tail_tile[warp] = tile;
                    } else if (ended) {
                        last_warp[tile] = warp;
                        if (u + 1 < u1) first_warp[tile + 1] = warp;
                    }
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
            at = 0;
            begun = true;
            ++tile;
        }
        __syncthreads();

        // ------------------------------------------------------------ the warps' sums, then the cluster's, then Y
        const int c = lane & 15, half = lane >> 4;       // a row of the tile; one of two tokens
        auto finish = [&](int j, int m, bool mine, float v) {
            v *= CodeScale<T>::back;
            const int n = ((r * p.round_tiles + j) * clusters + cluster) * kOut + c % kOut;
            if constexpr (GATED) {
                const float u = __shfl_down_sync(0xffffffffu, v, 8);       // the column's other sum
                if (mine && c < 8 && n < p.n) static_cast<T*>(p.y)[(int64_t)m * p.ldy + n] = (T)(activate(p.act, v) * u);
            } else if (mine && n < p.n) {
                static_cast<T*>(p.y)[(int64_t)m * p.ldy + n] = (T)v;
            }
        };
        if (KS == 1) {
            // tiles that a run begins and later ones end, two tokens of one at a time
            const int pairs_log = max(0, p.tokens_log - 1);
            for (int q = warp; q < W << pairs_log; q += W) {
                const int w = q >> pairs_log, j = tail_tile[w], m = 2 * (q - (w << pairs_log)) + half;
                if (j < 0) continue;
                const bool mine = m < p.tokens;
                float v = 0.f;
                if (mine) {
                    v = sums[((2 * w + 1) * kTokens + m) * kInt4Pitch + c];
                    const int end = (j + 1) * s_count;
                    for (int o0 = w + 1; o0 < W && units_to(all, o0) < end; o0 += 4)
#pragma unroll
                        for (int o = o0; o < o0 + 4; ++o) {
                            const int from = units_to(all, o);
                            if (o < W && from < end && from < units_to(all, o + 1)) v += sums[(2 * o * kTokens + m) * kInt4Pitch + c];
                        }
                }
                finish(j, m, mine, v);
            }
            return;
        }
        // The first slot of tile j is its first warp's; warps without units have none.
        auto add_warps = [&](int j, int m, int c) {
            float v = 0.f;
            for (int w = first_warp[j]; w <= last_warp[j]; ++w)
                if (units_to(all, w) < units_to(all, w + 1)) v += round_sums[((w + j) * kTokens + m) * kInt4Pitch + c];
            return v;
        };
        const int rows = count << p.tokens_log;       // tile j's token m is row j << tokens_log | m
        // in the place of the first warp's sums; each is read and written by one thread
        for (int q = 2 * warp + half; q < rows; q += 2 * W) {
            const int j = q >> p.tokens_log, m = q & ((1 << p.tokens_log) - 1);
            if (m < p.tokens && first_warp[j] < last_warp[j]) round_sums[((first_warp[j] + j) * kTokens + m) * kInt4Pitch + c] = add_warps(j, m, c);
        }
        cluster_sync();
        for (int q0 = 2 * warp; (q0 << p.k_split_log) < rows; q0 += 2 * W) {
            const int q = ((q0 + half) << p.k_split_log) + rank, j = q >> p.tokens_log, m = q & ((1 << p.tokens_log) - 1);
            const bool mine = q < rows && m < p.tokens;
            float v = 0.f;
            if (mine) {
                // the CTAs' parts of K may differ by a stage, and so the places of their sums
                for (int o = 0; o < KS; ++o) {
                    const int so = (int)(((int64_t)stages * (o + 1)) >> p.k_split_log) - (int)(((int64_t)stages * o) >> p.k_split_log);
                    const int w = so == s_count ? first_warp[j] : (W * (j * so + 1) - 1) / (count * so);
                    float s;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(s)
                                 : "r"(map_to_cta(smem_u32(round_sums + ((w + j) * kTokens + m) * kInt4Pitch + c), (uint32_t)o)));
                    v += s;
                }
            }
            finish(j, m, mine, v);
        }
        // A round's sums are written over two rounds on, when everyone has passed the barrier after them once more.
    }
    cluster_sync_relaxed();     // peers have read this CTA's sums
}

template <typename T, int VEC, int NB, bool GATED>
static cudaError_t launch_int4_as(const Int4Params& p, cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    auto kern = int4_matmul_kernel<T, VEC, NB, GATED>;
    const cudaError_t e = ensure_smem_limit(kern, (size_t)p.smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.grid);
    cfg.blockDim = dim3(32u << p.warps_log);
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

// How many clusters of 2^k_split_log CTAs the device holds at once, `per_sm` CTAs an SM by their shared memory.
template <typename T>
static cudaError_t resident_int4(int k_split_log, int per_sm, int* clusters) {
    auto kern = int4_matmul_kernel<T, 4, 1, false>;
    const size_t smem = (size_t)kInt4Room / per_sm;
    static std::atomic<int> smem_set[kMaxDevices];
    const cudaError_t e = ensure_smem_limit(kern, kInt4Room, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1u << k_split_log);
    cfg.blockDim = dim3((unsigned)kInt4MaxThreads / per_sm);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << k_split_log;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
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
