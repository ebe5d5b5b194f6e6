// lora_skinny.cu -- the projection with adapters (lora.cu) when it has few
// output tiles: decode batches and other short products, where the time is
// the stream of W and every SM has to take part in it.
//
// One cluster of 1, 2 or 4 CTAs computes one (128 tokens x tile_n) tile of
// Y, its CTAs splitting K and the tile's adapter steps evenly: each streams its
// share of X and W through a TMA ring and accumulates with tcgen05.mma into its
// own tensor memory, then the fp32 sums are added through distributed shared
// memory in rank order and every CTA of the cluster writes its part of the
// tile.  Against a split through global memory (partial tiles, flags, one
// finisher) the join costs a few hundred nanoseconds instead of microseconds
// and the adapter steps are shared out too (96 tokens x 4096 x 4096, 80
// adapters: 17.5 us here, 31.6 in the persistent kernel; 4 tokens: 11.0 and
// 21.5).  W comes by TMA: with asynchronous 16-byte copies by four warps the
// 96 tokens took 2.4 us longer.
//
// Only the tokens that exist are loaded: X boxes are round_up(tokens, 8) rows
// high, and the matrix instruction's other rows read whatever lies behind
// them in shared memory -- a row of the accumulator depends on its own row of
// X alone, and rows past the last token are never stored.
//
// Roles: warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps 2..5
// first list the tile's adapters (the producer then fetches their B before T is
// ready) and at the end read the accumulator (32 rows each).  Waits are bounded
// as in the persistent kernel; on expiry the CTA records GEMM_ERR_TIMEOUT and
// still takes part in the cluster's barriers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "elem.cuh"
#include "lora_list.cuh"
#include "lora_repair.cuh"
#include "lora_skinny.h"
#include "pipeline.cuh"
#include "ptx.cuh"
#include "serving_host.h"

namespace dgb {

constexpr int kSkinnyThreads = 192;

template <int OUT>
__global__ void __launch_bounds__(kSkinnyThreads, 1) skinny_kernel(const __grid_constant__ SkinnyParams p,
                                                                   const __grid_constant__ LoraTail tail) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[2 * kSkinnyMaxStages + 3];
    __shared__ AdapterList adapters;
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t abort_word;
    volatile uint32_t* abort_flag = &abort_word;

    const int S = p.stages;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * S, done_bar = empty0 + 8u * S, list_bar = done_bar + 8u;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int KS = p.k_split;
    const int r = KS > 1 ? (int)cluster_ctarank() : 0;
    const int n0 = (int)(blockIdx.x / KS) * p.tile_n, mb = blockIdx.y, m0 = mb * 128;
    const uint64_t tmo = p.timeout_ns;
    const uint32_t tile_id = blockIdx.y * gridDim.x + blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, 1);
        }
        mbar_init(done_bar, 1);
        mbar_init(list_bar, 4);
        abort_word = 0u;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tensormap(&p.tmap_x);
        prefetch_tensormap(&p.tmap_w);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(&tmem_slot), (uint32_t)p.tmem_cols);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // The kernel before this one computes T and waited for its own predecessors before this launch could start, so X and
    // W are complete; only the adapter steps wait for it (as in the persistent kernel).
    griddep_launch_dependents();

    const int kb0 = p.k_blocks * r / KS, kb1 = p.k_blocks * (r + 1) / KS;
    const uint32_t x_bytes = (uint32_t)p.box_m * 128u, stage_bytes = x_bytes + (uint32_t)p.tile_n * 128u;
    const uint32_t step_b = (uint32_t)p.tile_n * kTailRowBytes;

    if (warp == 0) {
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool aborted = false;
        const bool issuer = elect_one();
        auto take = [&]() {
            if (!wait_phase_warp<false, true>(empty0 + 8u * stage, phase ^ 1u, abort_flag, tmo, p.status, kRoleProducer, stage, tile_id)) {
                aborted = true;
                return false;
            }
            return true;
        };
        auto next = [&]() {
            __syncwarp();
            ++issued;
            if (++stage == S) { stage = 0; phase ^= 1u; }
        };
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!take()) break;
            if (issuer) {
                const uint32_t fb = full0 + 8u * stage, sx = smem_u32(ring + (size_t)stage * stage_bytes);
                mbar_arrive_expect_tx(fb, stage_bytes);
                tma_load_2d(sx + x_bytes, &p.tmap_w, fb, kb * 64, n0);
                tma_load_2d(sx, &p.tmap_x, fb, kb * 64, m0);
            }
            next();
        }
        // The adapter steps.  B does not depend on the kernel before: the first ring of groups gets its B, then, after that
        // kernel, its T; later groups both at once.
        bool waited = false;
        if (!aborted && wait_phase_warp<false>(list_bar, 0, abort_flag, tmo, p.status, kRoleProducer, 0, tile_id)) {
            const int total = adapters.count * tail.steps, groups = (total + 3) / 4;
            const int g0 = groups * r / KS, g1 = groups * (r + 1) / KS;
            const int early = min(g1 - g0, S), stage0 = stage;
            int begun = 0;        // groups that have their B on the way
            auto load_t = [&](int g, int st) {
                if (issuer) tma_load_3d(smem_u32(ring + (size_t)st * stage_bytes), &tail.tmap_t, full0 + 8u * st, g * 64, 0, mb);
            };
            for (int g = g0; g < g1; ++g) {
                if (g == g0 + early) {
                    griddep_wait();
                    waited = true;
                    for (int i = 0; i < early; ++i) load_t(g0 + i, (stage0 + i) % S);
                }
                if (!take()) break;
                const uint32_t fb = full0 + 8u * stage, sb = smem_u32(ring + (size_t)stage * stage_bytes) + x_bytes;
                const int n16 = min(4, total - 4 * g);
                if (issuer) {
                    mbar_arrive_expect_tx(fb, x_bytes + n16 * step_b);
                    for (int j = 0; j < n16; ++j) {
                        const int s = 4 * g + j, slot = s / tail.steps, c = s - slot * tail.steps;
                        tma_load_3d(sb + j * step_b, &tail.tmap_b, fb, (c % tail.b_steps) * 16, n0, adapters.list[slot]);
                    }
                }
                if (waited) load_t(g, stage);
                ++begun;
                next();
            }
            if (!waited) {
                griddep_wait();
                waited = true;
                for (int i = 0; i < begun; ++i) load_t(g0 + i, (stage0 + i) % S);
            }
        } else {
            aborted = true;
        }
        if (!waited) griddep_wait();
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
        bool aborted = false, first = true;
        const bool issuer = elect_one();
        auto take = [&]() {
            if (!wait_phase_warp<false>(full0 + 8u * stage, phase, abort_flag, tmo, p.status, kRoleMma, stage, tile_id)) {
                aborted = true;
                return false;
            }
            return true;
        };
        auto next = [&]() {
            __syncwarp();
            first = false;
            if (++stage == S) { stage = 0; phase ^= 1u; }
        };
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!take()) break;
            if (issuer) {
                tc_fence_after();
                const uint32_t sx = smem_u32(ring + (size_t)stage * stage_bytes);
                const uint64_t da = smem_desc_sw128(sx), db = smem_desc_sw128(sx + x_bytes);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_f16<1>(tmem, da + 2u * kk, db + 2u * kk, p.idesc, !first || kk != 0);
                mma_commit(empty0 + 8u * stage);
            }
            next();
        }
        if (!aborted) {
            if (!wait_phase_warp<false>(list_bar, 0, abort_flag, tmo, p.status, kRoleMma, 0, tile_id)) aborted = true;
            const int total = adapters.count * tail.steps, groups = (total + 3) / 4;
            const int g1 = groups * (r + 1) / KS;
            for (int g = groups * r / KS; !aborted && g < g1; ++g) {
                if (!take()) break;
                if (issuer) {
                    tc_fence_after();
                    const uint32_t sx = smem_u32(ring + (size_t)stage * stage_bytes);
                    const uint64_t da = smem_desc_sw128(sx), db = smem_desc_sw32(sx + x_bytes);
                    const int n16 = min(4, total - 4 * g);
                    for (int j = 0; j < n16; ++j) mma_f16<1>(tmem, da + 2u * j, db + (uint64_t)j * (step_b / 16u), p.idesc, 1u);
                    mma_commit(empty0 + 8u * stage);
                }
                next();
            }
        }
        if (issuer) {
            // every MMA issued so far (on the abort path too) completes here
            mma_commit(done_bar);
            if (aborted) wait_phase_drain(done_bar, 0, tmo);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ the tile's adapters
        find_adapters(p.adapter, p.adapters, p.M, m0, 128, adapters, (int32_t*)nullptr, 0, 0, (int)threadIdx.x - 64, 128,
                      [] { asm volatile("bar.sync 1, 128;" ::: "memory"); });
        if (lane == 0) mbar_arrive(list_bar);
        // ------------------------------------------------------------ accumulator to shared memory
        const int wq = warp & 3;      // tensor-memory lanes [32 wq, +32)
        bool ok = wait_phase_warp<false>(done_bar, 0, abort_flag, tmo, p.status, kRoleEpilogue, 0, tile_id);
        tc_fence_after();
        const int row = wq * 32 + lane;
        // the ring is idle: every copy has been consumed by an MMA and every MMA is complete
        float* sums = reinterpret_cast<float*>(ring);
        if (ok && m0 + wq * 32 < p.M) {
            for (int c = 0; c < p.tile_n; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tmem + ((uint32_t)(wq * 32) << 16) + c, v);
                tmem_wait_ld();
                tmem_reg_fence(v);
                if (m0 + row < p.M) {
                    float4* dst = reinterpret_cast<float4*>(sums + (size_t)row * p.sum_pitch + c);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
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
        const int rows = min(128, p.M - m0);
        const int pieces = p.tile_n / 4, all = rows * pieces;
        const int i1 = all * (r + 1) / KS;
        const uint32_t mine = smem_u32(ring);
        float probe = 0.f;
        constexpr int kAhead = 4;      // pieces of a thread whose loads are in flight
        for (int i0 = all * r / KS + (int)threadIdx.x; i0 < i1; i0 += kAhead * kSkinnyThreads) {
            float4 x[kAhead][kSkinnyMaxSplit];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kSkinnyThreads;
                if (i >= i1) break;
                const uint32_t at = mine + (uint32_t)(i / pieces * p.sum_pitch + i % pieces * 4) * 4u;
#pragma unroll
                for (int q = 0; q < kSkinnyMaxSplit; ++q)
                    if (q < KS) x[u][q] = load_cluster_f4(KS > 1 ? map_to_cta(at, (uint32_t)q) : at);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kSkinnyThreads;
                if (i >= i1) break;
                const int row = i / pieces, c = (i - row * pieces) * 4;
                float4 v = x[u][0];
#pragma unroll
                for (int q = 1; q < kSkinnyMaxSplit; ++q) {
                    if (q >= KS) break;
                    v.x += x[u][q].x;
                    v.y += x[u][q].y;
                    v.z += x[u][q].z;
                    v.w += x[u][q].w;
                }
                const int n = n0 + c;
                if (n >= p.N) continue;
                const int64_t o = (int64_t)(m0 + row) * p.ldy + n;
                const float f[4] = {v.x, v.y, v.z, v.w};
                probe = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, probe))));
                if constexpr (OUT == GEMM_F32) {
                    float* y = static_cast<float*>(p.y) + o;
                    if (n + 4 <= p.N) {
                        *reinterpret_cast<float4*>(y) = v;
                    } else {
                        for (int j = 0; n + j < p.N; ++j) y[j] = f[j];
                    }
                } else {
                    uint16_t* y = static_cast<uint16_t*>(p.y) + o;
                    const uint2 w = make_uint2(pack2<OUT>(f[0], f[1]), pack2<OUT>(f[2], f[3]));
                    if (n + 4 <= p.N) {
                        *reinterpret_cast<uint2*>(y) = w;
                    } else {
                        const uint16_t h[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
                        for (int j = 0; n + j < p.N; ++j) y[j] = h[j];
                    }
                }
            }
        }
        if (probe != 0.f)       // one of this thread's values is not finite
            for (int i = all * r / KS + (int)threadIdx.x; i < i1; i += kSkinnyThreads) {
                const int row = i / pieces, n = n0 + (i - row * pieces) * 4;
                repair_row<OUT>(tail, m0 + row, mb, n, min(n + 4, p.N),
                                static_cast<uint8_t*>(p.y) + ((int64_t)(m0 + row) * p.ldy + n) * (OUT == GEMM_F32 ? 4 : 2));
            }
    }
    if (KS > 1) cluster_sync_relaxed(); else __syncthreads();     // peers have read this CTA's sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem, (uint32_t)p.tmem_cols);
    }
}

template <int OUT>
static cudaError_t launch_typed(const SkinnyParams& p, const LoraTail& tail, dim3 grid, size_t smem, cudaStream_t stream) {
    auto kern = skinny_kernel<OUT>;
    static std::atomic<int> smem_set[kMaxDevices];
    cudaError_t e = ensure_smem_limit(kern, smem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kSkinnyThreads);
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
    return cudaLaunchKernelEx(&cfg, kern, p, tail);
}

cudaError_t launch_skinny(const SkinnyParams& p, const LoraTail& tail, int dtype_y, dim3 grid, size_t smem, cudaStream_t stream) {
    switch (dtype_y) {
    case GEMM_F32: return launch_typed<GEMM_F32>(p, tail, grid, smem, stream);
    case GEMM_BF16: return launch_typed<GEMM_BF16>(p, tail, grid, smem, stream);
    case GEMM_F16: return launch_typed<GEMM_F16>(p, tail, grid, smem, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dgb
