// int4_matmul.h -- products of a few tokens with 4-bit weights: launch parameters (int4_matmul.cuh; internal).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace dgb {

constexpr int kInt4TokensMax = 16;
constexpr int kInt4RowsMax = 1 << 30;     // of Y's columns: tiles past the last are counted too
constexpr int kInt4Warps = 8;
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
    int32_t k_warps_log;        // warps of a CTA that share a tile's part of K
    int32_t rounds;             // tiles that a warp goes through
    int32_t grid, smem;
};

cudaError_t launch_int4_bf16(const Int4Params& p, bool gated, cudaStream_t stream);
cudaError_t launch_int4_f16(const Int4Params& p, bool gated, cudaStream_t stream);

}  // namespace dgb
