// gated_few.h -- launch parameters of the gated pair of projections when it has few tiles (gated_few.cu; internal).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "serving_host.h"

namespace dgb {

constexpr int kGatedFewMaxStages = 16;
constexpr int kGatedFewMaxSplit = 4;    // CTAs of a cluster

struct GatedFewParams {
    CUtensorMap tmap_x;       // X: (K, tokens), box (64, box_m), 128-byte swizzle
    CUtensorMap tmap_w;       // W: (K, 2 features), box (64, half), 128-byte swizzle
    void* y;
    void* gate;               // both sums for the backward pass, or NULL
    void* up;
    int64_t ldy, ld_gate_up;
    gemm_device_error_t* status;
    uint64_t timeout_ns;
    int32_t M, features;
    int32_t k_blocks;         // 64-element blocks of K
    int32_t box_m;            // rows of X per tile: round_up(tokens, 8)
    int32_t half;             // columns of the output per tile: a multiple of 8 up to 128
    int32_t stages, tmem_cols;
    int32_t k_split;          // CTAs of a cluster
    int32_t sum_pitch;        // floats between rows of the sums laid over the ring: 2 half + 4
    int32_t act;
    uint32_t idesc;
};

// grid: column tiles x k_split; clusters of k_split.
cudaError_t launch_gated_few(const GatedFewParams& p, int dtype, dim3 grid, size_t smem, cudaStream_t stream);

// How many clusters of k_split CTAs, an SM's shared memory each, the device holds at once.
cudaError_t gated_few_max_clusters(int dtype, int k_split, const DeviceFacts& dev, int* clusters);

}  // namespace dgb
