// few_tokens.cuh -- Y = X W^T for up to 16 tokens, W in 16 bits or in 4 bits with
// group scales, alone or as a gated pair: the time is one stream over W.
//
// A warp multiplies 16 rows of W (of a gated pair: 8 gates and the 8 columns they
// multiply) by 8 or 16 tokens with 16 x 8 x 16 matrix instructions, W on the 16-row
// side, straight from global memory: which 16 of K's elements one instruction takes is
// free as long as both operands agree, so each lane loads consecutive ones of its two
// rows, 256 bytes of a row per four lanes and stage, and no weight passes through
// shared memory.  X lies there, laid out once per block so that a lane's part of an
// instruction pair is one 16-byte load.  A block's warps share a tile's K (several
// tiles where K is short); a block goes from tile to tile with the next stage's weights
// on the way, across tiles too, and two blocks an SM cover each other's joins.  The CTAs
// of a cluster share K when there are few tiles or X does not fit.  All sums are fp32 in
// a fixed order, so a column's sum never depends on timing.
//
// 4-bit codes become the 16-bit integers q - z exactly: a code in the low bits of
// the float 2^7 (bf16) or 2^10 (f16) reads 128 + q or 1024 + q, and subtracting
// 128 + z is exact.  A chunk of K that lies in one group is summed first, in fp32,
// and then multiplied by the group's scale in fp32: nothing is rounded to 16 bits.
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "activation.cuh"
#include "common.cuh"
#include "elem.cuh"
#include "few_tokens.h"

namespace dgb {

constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewPitch = 17;           // floats between tokens of a warp's sums: 16 rows

// `magic`: 2^7 (bf16) or 2^10 (f16) twice, a code in whose low bits is added to it.  `minus`: the same, negated, as 16 bits.
// `plus`: a + b of both halves, exact here.
template <typename T>
struct CodeBits;
template <>
struct CodeBits<__nv_bfloat16> {
    static constexpr uint32_t magic = 0x43004300u, minus = 0xC300u;
    static __device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0x3F803F80u), "r"(b));
        return r;
    }
};
template <>
struct CodeBits<__half> {
    static constexpr uint32_t magic = 0x64006400u, minus = 0xE400u;
    static __device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};

// Codes j and j + 4 of a word, as two floats `magic` + code: one shift and one three-operand operation (left to the compiler it
// becomes two of those and the shift between them, and bitwise operations run at half rate).
template <typename T, int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t word) {
    uint32_t s = word, r;
    if constexpr (J > 0) asm("shr.u32 %0, %1, %2;" : "=r"(s) : "r"(word), "n"(4 * J));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(s), "r"(0x000F000Fu), "r"(CodeBits<T>::magic));      // (s & mask) | magic
    return r;
}

// `bytes` (may be over 16 or negative) bytes of p's 16, the rest as zeros; elements of 2 bytes.
__device__ __forceinline__ uint4 load_clipped16(const void* p, int bytes) {
    if (bytes >= 16) return __ldg(static_cast<const uint4*>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (2 * i + 2 <= bytes) w[i >> 1] |= (uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t load_clipped4(const void* p, int bytes) {
    uint32_t w = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < bytes) w |= (uint32_t)__ldg(static_cast<const uint8_t*>(p) + i) << (8 * i);
    return w;
}
// weights: read once by the whole grid
__device__ __forceinline__ uint4 load_once16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <typename T, int VEC, int NB, bool GATED>
__global__ void __launch_bounds__(kFewThreads, 2) few_tokens_kernel(const __grid_constant__ FewParams p) {
    constexpr bool kCodes = VEC > 0;
    constexpr int kWords = kCodes ? VEC : 4;                // consecutive words of a row that a lane takes
    constexpr int kChunks = kFewRowBytes / 16 / kWords;     // of a stage: 4 lanes x kWords words of a row each
    constexpr int kRowWords = kChunks * kWords;             // of a stage and lane
    constexpr int kPerWord = kCodes ? 8 : 2;                // elements of K
    constexpr int kChunkK = 4 * kWords * kPerWord, kStageK = kChunks * kChunkK;
    constexpr int kVectors = kCodes ? VEC : 1;              // eight consecutive elements of x that a lane takes per chunk
    constexpr int kStageVectors = kChunks * kVectors;
    constexpr int kTokens = 8 * NB;
    constexpr int kOut = GATED ? 8 : 16;                    // columns of Y of a tile

    extern __shared__ uint4 few_smem[];
    float* sums = reinterpret_cast<float*>(few_smem);       // [2][warp][token][kFewPitch]
    uint4* x_smem = few_smem + 2 * kFewWarps * kTokens * kFewPitch / 4;         // [stage][vector][NB][lane]

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int KS = 1 << p.k_split_log, rank = KS > 1 ? (int)cluster_ctarank() : 0;
    const int KW = 1 << p.k_warps_log, share = warp & (KW - 1), sub = warp >> p.k_warps_log;    // of the warps that share a tile; which of the block's tiles
    const int per_round = kFewWarps >> p.k_warps_log;                   // tiles of a block at a time
    const int clusters = (int)gridDim.x >> p.k_split_log, cluster = (int)blockIdx.x >> p.k_split_log;

    const int stages = (p.k + kStageK - 1) / kStageK, whole = p.k / kStageK;
    const int s0 = (int)(((int64_t)stages * rank) >> p.k_split_log), s_count = (int)(((int64_t)stages * (rank + 1)) >> p.k_split_log) - s0;
    const int per_tile = (s_count + KW - 1) >> p.k_warps_log;           // stages of a warp in a tile
    const int own = s_count > share ? (s_count - share + KW - 1) >> p.k_warps_log : 0;     // of which this one has so many, the rest lie past the end
    const int tiles = (p.n + kOut - 1) / kOut;
    const int rounds = p.rounds;
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
            from[i] = static_cast<const uint8_t*>(p.w) + row_of(tile, i) * p.ldw_bytes + (int64_t)(s0 + share) * kFewRowBytes + 4 * kWords * t;
    };
    // The lines of the stage that is loaded next into L2, four lanes a row pair's four lines: its loads are issued a stage later and
    // used a stage after that, which alone does not cover DRAM's latency under load.
    auto prefetch = [&] {
        if (load_tile && load_at < own && s0 + share + (load_at << p.k_warps_log) < whole)
            asm volatile("prefetch.global.L2 [%0];" ::"l"((t & 1 ? from[1] : from[0]) + (128 * (t >> 1) - 4 * kWords * t)));
    };
    auto load = [&](uint32_t (&w)[2][kRowWords]) {
        if (load_tile && load_at < own) {
            const int stage = s0 + share + (load_at << p.k_warps_log);
            if (stage < whole) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const uint8_t* q = from[i] + c * (16 * kWords);
                        if constexpr (kWords == 4) {
                            const uint4 v = load_once16(q);
                            w[i][4 * c] = v.x;
                            w[i][4 * c + 1] = v.y;
                            w[i][4 * c + 2] = v.z;
                            w[i][4 * c + 3] = v.w;
                        } else if constexpr (kWords == 2) {
                            const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
                            w[i][2 * c] = v.x;
                            w[i][2 * c + 1] = v.y;
                        } else {
                            w[i][c] = __ldg(reinterpret_cast<const uint32_t*>(q));
                        }
                    }
            } else {
                const int left = (kCodes ? p.k / 2 : 2 * p.k) - stage * kFewRowBytes - 4 * kWords * t;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < kRowWords; ++j) {
                        const int o = (j / kWords) * (16 * kWords) + 4 * (j % kWords);
                        w[i][j] = load_clipped4(from[i] + o, left - o);
                    }
            }
        }
        if (++load_at < per_tile) {
#pragma unroll
            for (int i = 0; i < 2; ++i) from[i] += KW * kFewRowBytes;
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
    constexpr int kFactors = VEC == 1 ? 4 : VEC == 2 ? 2 : 1;
    int look_round = 0, look_at = 0;
    bool look_tile = false;
    uint16_t scale_next[2][kFactors] = {};
    uint8_t zero_next[2][kFactors] = {};
    int in_group_next = 0;      // where in its group the stage begins, in 32s
    const uint16_t* scale_row[2];
    const uint8_t* zero_row[2];
    const int last_group = kCodes ? (p.k - 1) / p.group : 0, group_units = kCodes ? p.group / 32 : 1;
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
        if constexpr (kCodes) {
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
        }
    };

    uint32_t now[2][kRowWords], next[2][kRowWords];
    set_rows();
    prefetch();         // while the kernel before this one may still run: it returns nothing, so it does not matter who writes W
    griddep_wait();
    griddep_launch_dependents();
    load(next);
    if constexpr (kCodes) set_looks();
    look();
    // X of this CTA's part of K, a warp an instruction pair's 32 lanes at a time: zeros past K and past the last token
    constexpr int kBatch = 4;       // loads of a thread on the way
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int m = nb * 8 + g, k_left = m < p.tokens ? p.k - s0 * kStageK - 8 * kVectors * t : 0;
        const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)min(m, p.tokens - 1) * p.ldx + s0 * kStageK + 8 * kVectors * t;
        for (int v0 = warp; v0 < s_count * kStageVectors; v0 += kBatch * kFewWarps) {
            uint4 q[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int v = v0 + b * kFewWarps, k = v / kVectors * kChunkK + v % kVectors * 8;
                q[b] = make_uint4(0u, 0u, 0u, 0u);
                if (v < s_count * kStageVectors && k < k_left) q[b] = load_clipped16(x + k, 2 * (k_left - k));
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int v = v0 + b * kFewWarps;
                if constexpr (kCodes)      // elements j and j + 4 of a word of codes lie 16 bits apart
                    q[b] = make_uint4(__byte_perm(q[b].x, q[b].z, 0x5410), __byte_perm(q[b].x, q[b].z, 0x7632),
                                      __byte_perm(q[b].y, q[b].w, 0x5410), __byte_perm(q[b].y, q[b].w, 0x7632));
                if (v < s_count * kStageVectors) x_smem[(v * NB + nb) * 32 + lane] = q[b];
            }
        }
    }
    __syncthreads();

    constexpr int kChains = NB == 1 ? 2 : 1;        // an accumulator's instructions wait for one another: two take turns
    float acc[kChains][NB][4];
#pragma unroll
    for (int q = 0; q < kChains; ++q)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[q][nb][i] = 0.f;
    int r = 0, at = 0;
    bool tile_here = tile_of(0) < tiles;
    const int all_stages = rounds * per_tile;
    for (int f = 0; f < all_stages; ++f) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kRowWords; ++j) now[i][j] = next[i][j];
        load(next);
        uint32_t factor[2][kFactors];           // a group's scale and, in the upper half, what makes its codes integers
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < kFactors; ++h)
                factor[i][h] = (uint32_t)scale_next[i][h] | ((uint32_t)zero_next[i][h] << 16) | (CodeBits<T>::minus << 16);
        int in_group = in_group_next;
        look();
        if (tile_here && at < own) {
            const int in = share + (at << p.k_warps_log);
            const uint4* x = x_smem + (size_t)in * (kStageVectors * NB * 32) + lane;
            const int chunks = kCodes ? (p.k - (s0 + in) * kStageK + kChunkK - 1) / kChunkK : kChunks;     // that K reaches
            int gi = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (kCodes && c >= chunks) break;
                const uint32_t* lo = now[0] + c * kWords;
                const uint32_t* hi = now[1] + c * kWords;
                if constexpr (!kCodes) {
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint4 q = x[(c * NB + nb) * 32];
                        mma_16816<T>(acc[0][nb], a0, q.x, q.y);
                        mma_16816<T>(acc[kChains - 1][nb], a1, q.z, q.w);
                    }
                } else {
                    float part[kChains][NB][4];
                    float scale[2];
                    uint32_t less[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t mine = factor[i][0];
#pragma unroll
                        for (int h = 1; h < kFactors; ++h)
                            if (gi >= 4 * h) mine = factor[i][h];
                        const uint32_t f32 = __shfl_sync(0xffffffffu, mine, (lane & 28) | (gi & 3));
                        scale[i] = unpack2<T>(f32).x;
                        less[i] = __byte_perm(f32, 0u, 0x3232);
                    }
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        const uint32_t a0[4] = {CodeBits<T>::plus(code_pair<T, 0>(lo[v]), less[0]), CodeBits<T>::plus(code_pair<T, 0>(hi[v]), less[1]),
                                                CodeBits<T>::plus(code_pair<T, 1>(lo[v]), less[0]), CodeBits<T>::plus(code_pair<T, 1>(hi[v]), less[1])};
                        const uint32_t a1[4] = {CodeBits<T>::plus(code_pair<T, 2>(lo[v]), less[0]), CodeBits<T>::plus(code_pair<T, 2>(hi[v]), less[1]),
                                                CodeBits<T>::plus(code_pair<T, 3>(lo[v]), less[0]), CodeBits<T>::plus(code_pair<T, 3>(hi[v]), less[1])};
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const uint4 q = x[((c * VEC + v) * NB + nb) * 32];
                            if (v == 0) mma_16816_fresh<T>(part[0][nb], a0, q.x, q.y);
                            else mma_16816<T>(part[0][nb], a0, q.x, q.y);
                            if (v == 0 && kChains > 1) mma_16816_fresh<T>(part[kChains - 1][nb], a1, q.z, q.w);
                            else mma_16816<T>(part[kChains - 1][nb], a1, q.z, q.w);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < kChains; ++q)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[q][nb][i] = fmaf(scale[i >> 1], part[q][nb][i], acc[q][nb][i]);
                    in_group += kChunkK / 32;
                    if (in_group >= group_units) {
                        in_group -= group_units;
                        ++gi;
                    }
                }
            }
        }
        if (++at < per_tile) continue;
        at = 0;

        // ------------------------------------------------------------ a tile's end: the warps' sums, then the cluster's, then Y
        float* mine = sums + (r & 1) * (kFewWarps * kTokens * kFewPitch);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mine[(warp * kTokens + nb * 8 + 2 * t + (i & 1)) * kFewPitch + (i >> 1) * 8 + g] =
                    kChains == 1 ? acc[0][nb][i] : acc[0][nb][i] + acc[kChains - 1][nb][i];
                acc[0][nb][i] = acc[kChains - 1][nb][i] = 0.f;
            }
        // the tile's warps meet; a buffer is written again two rounds on, after all have met once more
        const int threads = 32 * KW, thread = share * 32 + lane;
        if (KW == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(threads) : "memory");
        float* tile_sums = mine + sub * KW * kTokens * kFewPitch;
        auto add_warps = [&](int m, int c) {
            float v = tile_sums[m * kFewPitch + c];
#pragma unroll 4
            for (int w = 1; w < KW; ++w) v += tile_sums[(w * kTokens + m) * kFewPitch + c];
            return v;
        };
        int m0 = 0, m1 = p.tokens;
        if (KS > 1) {
            // in the place of the first warp's sums; each is read and written by one thread
            for (int e = thread; e < p.tokens * 16; e += threads) tile_sums[e / 16 * kFewPitch + e % 16] = add_warps(e / 16, e % 16);
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
                const uint32_t part = smem_u32(tile_sums + m * kFewPitch + c);
                for (int o = 0; o < KS; ++o) {
                    float s;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(s) : "r"(map_to_cta(part, (uint32_t)o)));
                    v += s;
                }
            }
            const int n = tile_of(r) * kOut + c % kOut;
            const bool there = e < m1 * 16 && n < p.n;
            if constexpr (GATED) {
                const float u = __shfl_down_sync(0xffffffffu, v, 8);       // the column's other sum
                if (there && c < 8) {
                    if (p.gate) {
                        static_cast<T*>(p.gate)[(int64_t)m * p.ld_gate_up + n] = (T)v;
                        static_cast<T*>(p.up)[(int64_t)m * p.ld_gate_up + n] = (T)u;
                    }
                    static_cast<T*>(p.y)[(int64_t)m * p.ldy + n] = (T)(activate(p.act, v) * u);
                }
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
static cudaError_t launch_few_as(const FewParams& p, cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    auto kern = few_tokens_kernel<T, VEC, NB, GATED>;
    const cudaError_t e = ensure_smem_limit(kern, (size_t)p.smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.grid);
    cfg.blockDim = dim3(kFewThreads);
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
static cudaError_t launch_few_vec(const FewParams& p, bool gated, cudaStream_t stream) {
    if (p.tokens > 8) return gated ? launch_few_as<T, VEC, 2, true>(p, stream) : launch_few_as<T, VEC, 2, false>(p, stream);
    return gated ? launch_few_as<T, VEC, 1, true>(p, stream) : launch_few_as<T, VEC, 1, false>(p, stream);
}

template <typename T>
static cudaError_t launch_few(const FewParams& p, int vec, bool gated, cudaStream_t stream) {
    switch (vec) {
    case 0:     // the product of 16-bit weights alone is the library's own
        return p.tokens > 8 ? launch_few_as<T, 0, 2, true>(p, stream) : launch_few_as<T, 0, 1, true>(p, stream);
    case 1: return launch_few_vec<T, 1>(p, gated, stream);
    case 2: return launch_few_vec<T, 2>(p, gated, stream);
    default: return launch_few_vec<T, 4>(p, gated, stream);
    }
}

}  // namespace dgb
