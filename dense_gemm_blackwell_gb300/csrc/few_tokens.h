// few_tokens.h -- products of a few tokens with a weight matrix that is read once (few_tokens.cuh; internal).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace dgb {

constexpr int kFewTokensMax = 16;
constexpr int kFewWarps = 8;
constexpr int kFewRowBytes = 256;       // a stage: so many bytes of each of a tile's 16 rows

struct FewParams {
    const void* x;              // [tokens][k], 16 bits
    const void* w;              // 16-bit elements, or two 4-bit codes a byte
    const void* scales;         // 4-bit weights: [rows][groups], x's type
    const uint8_t* zeros;       // 4-bit weights: [rows][groups] or NULL (8)
    void* y;
    void* gate;                 // gated: both sums, rounded, or NULL
    void* up;
    int64_t ldx, ldw_bytes, ld_scales, ld_zeros, ldy, ld_gate_up;
    int32_t tokens, k, n;       // n: columns of y
    int32_t group;              // 4-bit weights: a multiple of 32
    int32_t act;                // gated
    // filled in by shape_few
    int32_t k_split_log;        // CTAs (one cluster) that share K
    int32_t k_warps_log;        // warps of a CTA that share a tile's part of K
    int32_t rounds;             // tiles that a warp goes through
    uint32_t group_magic;       // 4-bit weights: floor(2^32 / (group / 32)), at most 2^32 - 1
    int32_t grid, smem;
};

// vec: 0 = 16-bit weights; otherwise 4-bit words a lane loads at once (1, 2 or 4; group a multiple of 32 vec).  gated: w's
// first n rows are gates, the next n the columns they multiply.
cudaError_t launch_few_bf16(const FewParams& p, int vec, bool gated, cudaStream_t stream);
cudaError_t launch_few_f16(const FewParams& p, int vec, bool gated, cudaStream_t stream);

// Lays a product (tokens, n and k are set) on a device: false where its tokens do not fit shared memory.
bool shape_few(FewParams* p, bool gated, bool four_bits, int sms);

}  // namespace dgb
