// lora_skinny.h -- launch parameters of the few-tile projection with adapters (lora_skinny.cu; internal).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace dgb {

constexpr int kSkinnyMaxStages = 16;
constexpr int kSkinnyMaxSplit = 4;    // CTAs of a cluster

struct SkinnyParams {
    CUtensorMap tmap_x;       // X: (K, tokens), box (64, box_m), 128-byte swizzle
    CUtensorMap tmap_w;       // W: (K, N), box (64, tile_n), 128-byte swizzle
    void* y;
    int64_t ldy;
    const int32_t* adapter;   // [tokens]
    gemm_device_error_t* status;
    uint64_t timeout_ns;
    int32_t adapters;
    int32_t M, N;
    int32_t k_blocks;         // 64-element blocks of K
    int32_t box_m;            // rows of X per tile: round_up(min(tokens, 128), 8)
    int32_t tile_n, stages, tmem_cols;
    int32_t k_split;          // CTAs of a cluster
    int32_t sum_pitch;        // floats between rows of the sums laid over the ring: tile_n + 4
    uint32_t idesc;
};

// grid: (n tiles x k_split, m blocks); clusters of k_split along x.
cudaError_t launch_skinny(const SkinnyParams& p, const LoraTail& tail, int dtype_y, dim3 grid, size_t smem, cudaStream_t stream);

}  // namespace dgb
