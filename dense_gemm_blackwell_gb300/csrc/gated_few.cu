// gated_few.cu -- a gated pair of projections (gated.cu) for up to 128 tokens: the
// time is the stream of W and every SM has to take part in it.
//
// One cluster of 1, 2 or 4 CTAs computes one tile of all tokens x `half` columns,
// its CTAs splitting K evenly: each streams its share of X and of the tile's gates
// and ups through a TMA ring, accumulates with tcgen05.mma into its own tensor
// memory (gates in the first `half` columns, ups in the next), then the fp32 sums
// are added through distributed shared memory in rank order and every CTA of the
// cluster writes its part of act(gate) * up.  `half` is any multiple of 8: the
// columns are dealt out so that one wave of CTAs covers the device, which the
// persistent kernel's powers of two do not.
//
// Only the tokens that exist are loaded: X boxes are round_up(tokens, 8) rows
// high, and the matrix instruction's other rows read whatever lies behind them in
// shared memory -- a row of the accumulator depends on its own row of X alone, and
// rows past the last token are never stored.
//
// Bound by memory: 4 tokens x 4096 -> 2 x 12288 31.4-32.3 us, 6.3 TB/s (the bytes take
// 29.6); 1 token x 8192 -> 2 x 16384 79 us, all of the copy rate.  96 tokens 37-38 us:
// 2.3 times the bytes into shared memory, and sums that are joined behind the stream.
//
// Roles: warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps 2..5 read
// the accumulator (32 rows each); all join and store.  Waits are bounded as in the
// persistent kernel; on expiry the CTA records GEMM_ERR_TIMEOUT and still takes
// part in the cluster's barriers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "activation.cuh"
#include "common.cuh"
#include "gated_few.h"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace dgb {

constexpr int kGatedFewThreads = 192;

template <int OUT>
__global__ void __launch_bounds__(kGatedFewThreads, 1) gated_few_kernel(const __grid_constant__ GatedFewParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[2 * kGatedFewMaxStages + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t abort_word;
    volatile uint32_t* abort_flag = &abort_word;

    const int S = p.stages;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * S, done_bar = empty0 + 8u * S;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int KS = p.k_split;
    const int r = KS > 1 ? (int)cluster_ctarank() : 0;
    const int n0 = (int)(blockIdx.x / KS) * p.half;
    const uint64_t tmo = p.timeout_ns;
    const uint32_t tile_id = blockIdx.x;
    const int kb0 = p.k_blocks * r / KS, kb1 = p.k_blocks * (r + 1) / KS;
    const uint32_t x_bytes = (uint32_t)p.box_m * 128u, w_bytes = (uint32_t)p.half * 128u, stage_bytes = x_bytes + 2u * w_bytes;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, 1);
        }
        mbar_init(done_bar, 1);
        abort_word = 0u;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tensormap(&p.tmap_x);
        prefetch_tensormap(&p.tmap_w);
        // The ring's first W into L2 while the kernel before this one still runs: a prefetch returns nothing, so it does not
        // matter who writes W.
        for (int kb = kb0; kb < min(kb1, kb0 + S); ++kb) {
            tma_prefetch_2d(&p.tmap_w, kb * 64, n0);
            tma_prefetch_2d(&p.tmap_w, kb * 64, p.features + n0);
        }
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&tmem_slot), (uint32_t)p.tmem_cols);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool aborted = false;
        const bool issuer = elect_one();
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_phase_warp<false, true>(empty0 + 8u * stage, phase ^ 1u, abort_flag, tmo, p.status, kRoleProducer, stage, tile_id)) {
                aborted = true;
                break;
            }
            if (issuer) {
                const uint32_t fb = full0 + 8u * stage, sx = smem_u32(ring + (size_t)stage * stage_bytes);
                mbar_arrive_expect_tx(fb, stage_bytes);
                tma_load_2d(sx + x_bytes, &p.tmap_w, fb, kb * 64, n0);
                tma_load_2d(sx + x_bytes + w_bytes, &p.tmap_w, fb, kb * 64, p.features + n0);
                tma_load_2d(sx, &p.tmap_x, fb, kb * 64, 0);
            }
            __syncwarp();
            ++issued;
            if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (aborted) {
            // wait (bounded) for the copies still in flight into the ring
            const int n = issued < S ? issued : S;
            for (int i = 0; i < n; ++i) {
                if (stage == 0) { stage = S - 1; phase ^= 1u; } else { --stage; }
                wait_phase_drain(full0 + 8u * stage, phase, tmo);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        int stage = 0;
        uint32_t phase = 0;
        bool aborted = false;
        const bool issuer = elect_one();
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_phase_warp<false>(full0 + 8u * stage, phase, abort_flag, tmo, p.status, kRoleMma, stage, tile_id)) {
                aborted = true;
                break;
            }
            if (issuer) {
                tc_fence_after();
                const uint32_t sx = smem_u32(ring + (size_t)stage * stage_bytes);
                const uint64_t da = smem_desc_sw128(sx), db = smem_desc_sw128(sx + x_bytes);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_f16<1>(tmem, da + 2u * kk, db + 2u * kk, p.idesc, kb != kb0 || kk != 0);
                mma_commit(empty0 + 8u * stage);
            }
            __syncwarp();
            if (++stage == S) { stage = 0; phase ^= 1u; }
        }
        if (issuer) {
            // every MMA issued so far (on the abort path too) completes here
            mma_commit(done_bar);
            if (aborted) wait_phase_drain(done_bar, 0, tmo);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ accumulator to shared memory
        const int wq = warp & 3;      // tensor-memory lanes [32 wq, +32)
        const bool ok = wait_phase_warp<false>(done_bar, 0, abort_flag, tmo, p.status, kRoleEpilogue, 0, tile_id);
        tc_fence_after();
        const int row = wq * 32 + lane;
        // the ring is idle: every copy has been consumed by an MMA and every MMA is complete
        float* sums = reinterpret_cast<float*>(ring);
        if (ok && wq * 32 < p.M) {
            for (int c = 0; c < 2 * p.half; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + ((uint32_t)(wq * 32) << 16) + c, v);
                tmem_wait_ld();
                tmem_reg_fence(v);
                if (row < p.M) {
                    float4* dst = reinterpret_cast<float4*>(sums + (size_t)row * p.sum_pitch + c);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + 4 * j < 2 * p.half)
                            dst[j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]), __uint_as_float(v[4 * j + 2]),
                                                 __uint_as_float(v[4 * j + 3]));
                }
            }
        }
        tc_fence_before();
    }
    if (KS > 1) cluster_sync(); else __syncthreads();
    // ---------------------------------------------------------------- join and store: this CTA's share of the tile's rows
    {
        const int pieces = p.half / 4, all = p.M * pieces;
        const int i1 = all * (r + 1) / KS;
        const uint32_t mine = smem_u32(ring);
        constexpr int kAhead = 2;      // pieces of a thread whose loads are in flight
        for (int i0 = all * r / KS + (int)threadIdx.x; i0 < i1; i0 += kAhead * kGatedFewThreads) {
            float4 x[kAhead][2][kGatedFewMaxSplit];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kGatedFewThreads;
                if (i >= i1) break;
                const uint32_t at = mine + (uint32_t)(i / pieces * p.sum_pitch + i % pieces * 4) * 4u;
#pragma unroll
                for (int q = 0; q < kGatedFewMaxSplit; ++q)
                    if (q < KS) {
                        x[u][0][q] = load_cluster_f4(KS > 1 ? map_to_cta(at, (uint32_t)q) : at);
                        x[u][1][q] = load_cluster_f4(KS > 1 ? map_to_cta(at + 4u * p.half, (uint32_t)q) : at + 4u * p.half);
                    }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kGatedFewThreads;
                if (i >= i1) break;
                const int row = i / pieces, n = n0 + (i - row * pieces) * 4;
                if (n >= p.features) continue;      // features and columns come in fours
                float4 s[2];
#pragma unroll
                for (int kind = 0; kind < 2; ++kind) {
                    s[kind] = x[u][kind][0];
#pragma unroll
                    for (int q = 1; q < kGatedFewMaxSplit; ++q) {
                        if (q >= KS) break;
                        s[kind].x += x[u][kind][q].x;
                        s[kind].y += x[u][kind][q].y;
                        s[kind].z += x[u][kind][q].z;
                        s[kind].w += x[u][kind][q].w;
                    }
                }
                const float4 g = s[0], v = s[1];
                if (p.gate) {
                    const int64_t o = (int64_t)row * p.ld_gate_up + n;
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.gate) + o) = make_uint2(pack2<OUT>(g.x, g.y), pack2<OUT>(g.z, g.w));
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.up) + o) = make_uint2(pack2<OUT>(v.x, v.y), pack2<OUT>(v.z, v.w));
                }
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + (int64_t)row * p.ldy + n) =
                    make_uint2(pack2<OUT>(activate(p.act, g.x) * v.x, activate(p.act, g.y) * v.y),
                               pack2<OUT>(activate(p.act, g.z) * v.z, activate(p.act, g.w) * v.w));
            }
        }
    }
    if (KS > 1) cluster_sync_relaxed(); else __syncthreads();     // peers have read this CTA's sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem, (uint32_t)p.tmem_cols);
    }
}

static std::atomic<int> smem_set[2][kMaxDevices];      // of the kernel for f16 and for bf16

template <int OUT>
static cudaError_t launch_typed(const GatedFewParams& p, dim3 grid, size_t smem, cudaStream_t stream) {
    auto kern = gated_few_kernel<OUT>;
    cudaError_t e = ensure_smem_limit(kern, smem, smem_set[OUT == GEMM_BF16]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kGatedFewThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.k_split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t gated_few_max_clusters(int dtype, int k_split, const DeviceFacts& dev, int* clusters) {
    if (k_split == 1) {
        *clusters = dev.sms;
        return cudaSuccess;
    }
    auto kern = dtype == GEMM_BF16 ? gated_few_kernel<GEMM_BF16> : gated_few_kernel<GEMM_F16>;
    const size_t smem = (size_t)dev.smem_optin - 2048;
    const cudaError_t e = ensure_smem_limit(kern, smem, smem_set[dtype == GEMM_BF16]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)k_split);
    cfg.blockDim = dim3(kGatedFewThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)k_split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
}

cudaError_t launch_gated_few(const GatedFewParams& p, int dtype, dim3 grid, size_t smem, cudaStream_t stream) {
    return dtype == GEMM_BF16 ? launch_typed<GEMM_BF16>(p, grid, smem, stream) : launch_typed<GEMM_F16>(p, grid, smem, stream);
}

}  // namespace dgb
