// gated_epilogue.cuh -- the persistent kernel's epilogue for a gated pair of
// projections: act(gate) * up from an accumulator that holds both.
#pragma once

#include "activation.cuh"
#include "common.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace dgb {

// Roles, hand-back of accumulator parts, staging and stream-K partials are those of the plain epilogue (persistent.cuh).  A part
// (a whole tile up to 256 wide, or 256 columns of a 512-wide one) holds gates in its first half and ups in its second: a warp
// takes chunks of 64 output columns (128 bytes), 32 gates and 32 ups at a time, so that both sums of an element meet in one
// thread's registers and are never rounded before their product.  Bound by the tensor cores where the tiles are many: 8192 x 4096 -> 2 x
// 16384 bf16 1104 us in a graph, 2.0 PFLOP/s (1215 to 1226 in a loop of calls, when the power cap has set in), which is the plain
// product's rate; writing both sums out and reading them back would move 1.1 GB more, 158 us.  Keeping both sums for the backward
// pass: 1190 us where 1120 were measured beside it, 283 and 276 at 4096 x 4096 -> 2 x 8192.  One wave of tiles shows the
// epilogue: 777 x 1001 -> 2 x 1544 13.7 us, of which the product is 8.8.
template <int CG, int OUT>
__device__ __forceinline__ void gated_epilogue(const PersistentParams& p, const GatedTail& q, uint8_t* staging, uint32_t tmem_base,
                                               uint32_t tfull0, uint32_t tempty0, volatile uint32_t* abort_flag, uint32_t rank,
                                               int cluster_id, int num_clusters) {
    constexpr int kCols = 64;               // output columns of a chunk
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wq = warp & 3, second = (warp - 2) >> 2;
    const int TS = p.tmem_stages;
    const uint64_t tmo = p.timeout_ns;
    const uint64_t pol_d = l2_policy_evict_first();
    const bool stream_d = (p.l2_hints & kHintStreamD) != 0;
    uint8_t* buf = staging + (warp - 2) * kStagingBytes;
    auto tfull = [&](int a, int part) { return tfull0 + 8u * (2 * a + part); };
    auto tempty = [&](int a, int part) { return tempty0 + 8u * (2 * a + part); };
    const int parts = p.tile_n > 256 ? 2 : 1;
    const int part_cols = p.tile_n / parts, half_cols = part_cols / 2;      // columns of a part; of its gates
    const int chunks = half_cols / kCols;                                   // of a part
    const int split = (chunks + 1) / 2;                                     // the first warp of a lane quarter takes [0, split)
    const int c_lo = second ? split : 0, c_hi = second ? chunks : split;
    int acc = 0;
    uint32_t acc_phase = 0;
    WorkUnit u;
    for (int idx = 0; next_unit(p, cluster_id, num_clusters, idx, u); ++idx) {
        const int t = u.tile;
        int b, mb, nb;
        tile_coords(p, t, b, mb, nb);
        const uint32_t t_lane = tmem_base + ((uint32_t)(wq * 32) << 16) + (uint32_t)(acc * p.tile_n);
        const int m0 = mb * (128 * CG) + (int)rank * 128 + wq * 32;
        const int n0 = nb * (p.tile_n / 2);
        auto wait_part = [&](int pt) {
            const bool got = wait_phase_warp<false>(tfull(acc, pt), acc_phase, abort_flag, tmo, p.status, kRoleEpilogue, acc, t);
            tc_fence_after();
            return got;
        };
        auto release = [&](int pt) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<CG>(tempty(acc, pt));
        };
        auto part_base_of = [&](int s) { return (size_t)(s * CG + (int)rank) * 128 * p.tile_n / 4; };
        auto flag_of = [&](int s) { return p.sk_flags + (s * CG + (int)rank) * kEpilogueWarps + second * 4 + wq; };
        bool lost = false;

        if (u.role == kUnitContributor) {
            // the fp32 partial of both halves of this warp's chunks, for the finisher
            float4* part = reinterpret_cast<float4*>(p.sk_partials) + part_base_of(u.slot);
            for (int pt = 0; pt < parts; ++pt) {
                if (!wait_part(pt)) {
                    lost = true;
                    break;
                }
                if (c_lo >= c_hi) release(pt);
                for (int i = 2 * c_lo; i < 2 * c_hi; ++i)
#pragma unroll
                    for (int kind = 0; kind < 2; ++kind) {
                        const int col = pt * part_cols + kind * half_cols + 32 * i;
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(t_lane + col, r);
                        tmem_wait_ld();
                        tmem_reg_fence(r);
                        if (i + 1 == 2 * c_hi && kind == 1) release(pt);
                        float4* dst = part + sk_partial_index(p.tile_n, wq, col / 32, 0, lane);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[32 * j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                                                      __uint_as_float(r[4 * j + 3]));
                    }
            }
            if (lost) break;
            __threadfence();
            __syncwarp();
            if (lane == 0) store_release_gpu(flag_of(u.slot), sk_launch_epoch(p.sk_epoch));
            if (++acc == TS) { acc = 0; acc_phase ^= 1u; }
            continue;
        }

        const bool adds = u.role == kUnitFinisher;
        // a thread's row of sums `r` at accumulator column `col`: the contributors' partials, latest K range first
        auto add_partials = [&](uint32_t (&r)[32], int col) {
            for (int s = u.slot; s >= u.slot0; --s) {
                const float4* ps = reinterpret_cast<const float4*>(p.sk_partials) + part_base_of(s) +
                                   sk_partial_index(p.tile_n, wq, col / 32, 0, lane);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 v = __ldcg(ps + 32 * j);
                    r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + v.x);
                    r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + v.y);
                    r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + v.z);
                    r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + v.w);
                }
            }
        };
        // 128 bytes of each of this warp's 32 rows to columns [x, x + 64), through the staging buffer and a TMA store, which
        // leaves out what lies past the matrix (its columns are a multiple of 8: whole 16-byte granules)
        auto store_chunk = [&](const CUtensorMap* map, int x, const uint32_t (&w)[32]) {
            if (lane == 0) bulk_wait_group_read<0>();       // the buffer's previous store must have read it
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (stream_d) tma_store_2d_hint(map, smem_u32(buf), x, m0, pol_d);
                else tma_store_2d(map, smem_u32(buf), x, m0);
                bulk_commit_group();
            }
        };
        for (int pt = 0; pt < parts; ++pt) {
            if (!wait_part(pt)) {
                lost = true;
                break;
            }
            if (adds && pt == 0) {
                int got = 1;
                if (lane == 0)
                    for (int s = u.slot; s >= u.slot0 && got; --s)
                        got = wait_flag(flag_of(s), sk_launch_epoch(p.sk_epoch), abort_flag, tmo, p.status, kRoleEpilogue, s, t);
                got = __shfl_sync(0xffffffffu, got, 0);
                if (!got) {
                    for (int o = 0; o < parts; ++o) release(o);
                    lost = true;
                    break;
                }
                for (int s = u.slot; s >= u.slot0; --s) {
                    uint32_t v;   // every lane acquires the flags before reading the partials
                    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag_of(s)) : "memory");
                    (void)v;
                }
            }
            // chunks with a column and a row inside the output
            const int x0 = n0 + pt * half_cols;
            const int c_end = m0 < p.M ? min(c_hi, (q.features - x0 + kCols - 1) / kCols) : c_lo;
            if (c_lo >= c_end) release(pt);
            for (int c = c_lo; c < c_end; ++c) {
                const int x = x0 + c * kCols;
                uint32_t h[32];
                if (q.keep) {
                    // both sums for the backward pass, read once more: kept beside the outputs they would not fit the registers
#pragma unroll
                    for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int col = pt * part_cols + kind * half_cols + c * kCols + 32 * s;
                            uint32_t r[32];
                            tmem_ld_32x32b_x32(t_lane + col, r);
                            tmem_wait_ld();
                            tmem_reg_fence(r);
                            if (adds) add_partials(r, col);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                h[16 * s + i] = pack2<OUT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                        }
                        store_chunk(kind == 0 ? &q.tmap_gate : &q.tmap_up, x, h);
                    }
                }
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int col = pt * part_cols + c * kCols + 32 * s;
                    uint32_t rg[32], ru[32];
                    tmem_ld_32x32b_x32(t_lane + col, rg);
                    tmem_ld_32x32b_x32(t_lane + col + half_cols, ru);
                    tmem_wait_ld();
                    tmem_reg_fence(rg);
                    tmem_reg_fence(ru);
                    if (s == 1 && c + 1 == c_end) release(pt);
                    if (adds) {
                        add_partials(rg, col);
                        add_partials(ru, col + half_cols);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float g0 = __uint_as_float(rg[2 * i]), g1 = __uint_as_float(rg[2 * i + 1]);
                        const float u0 = __uint_as_float(ru[2 * i]), u1 = __uint_as_float(ru[2 * i + 1]);
                        h[16 * s + i] = pack2<OUT>(activate(q.act, g0) * u0, activate(q.act, g1) * u1);
                    }
                }
                store_chunk(&p.tmap_d, x, h);
            }
        }
        if (lost) break;
        if (++acc == TS) { acc = 0; acc_phase ^= 1u; }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
}

}  // namespace dgb
