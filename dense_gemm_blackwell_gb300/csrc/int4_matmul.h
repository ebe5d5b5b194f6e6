// int4_matmul.h -- products of a few tokens with 4-bit weights: launch parameters (int4_matmul.cuh; internal).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace dgb {

constexpr int kInt4TokensMax = 16;
constexpr int kInt4RowsMax = 1 << 30;     // of Y's columns: tiles past the last are counted too
constexpr int kInt4RoundTiles = 16;     // tiles of a cluster between two joins, at most; of 9 to 16 tokens half as many, of more
                                        // rounds than one half as many again
constexpr int kInt4Room = 224 * 1024;   // shared memory of an SM that its blocks take
constexpr int kInt4RowBytes = 256;      // a stage: so many bytes of each of a tile's 16 rows

struct Int4Params {
    const void* x;              // [tokens][k], 16 bits
    const void* w;              // two codes a byte
    const void* scales;         // [rows][groups], x's type
    const uint8_t* zeros;       // [rows][groups] or NULL (8)
    void* y;
    int64_t ldx, ldw_bytes, ld_scales, ld_zeros, ldy;
    int32_t tokens, k, n;       // n: columns of y; gated: w's first n rows are gates, the next n the columns they multiply
    int32_t group;              // a multiple of 32
    int32_t act;                // gated
    uint32_t group_magic;       // floor(2^32 / (group / 32)), at most 2^32 - 1
    int32_t tokens_log;         // tokens, rounded up to a power of two
    int32_t k_split_log;        // CTAs (one cluster) that share K
    int32_t warps_log;          // warps of a CTA: 8, two CTAs an SM, or 16
    int32_t round_tiles;        // tiles of a cluster between two joins; without clusters all of a CTA's
    int32_t slots;              // places of a warp's sums of a tile, of more rounds than one for two rounds
    int32_t grid, smem;
};

// Clusters of 2^k_split_log CTAs, `per_sm` CTAs an SM, that the device holds at once.
cudaError_t int4_resident(int k_split_log, int per_sm, int* clusters);
cudaError_t launch_int4_bf16(const Int4Params& p, bool gated, cudaStream_t stream);
cudaError_t launch_int4_f16(const Int4Params& p, bool gated, cudaStream_t stream);

}  // namespace dgb
