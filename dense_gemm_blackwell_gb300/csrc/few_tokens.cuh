// few_tokens.cuh -- Y = X W^T for up to 16 tokens, W in 16 bits or in 4 bits with
// group scales, alone or as a gated pair: the time is one stream over W.
//
// A warp multiplies two blocks of 16 rows of W (of a gated pair: gates and the
// columns they multiply) by 8 or 16 tokens with 16 x 8 x 16 matrix instructions,
// W on the 16-row side, straight from global memory: which 16 of K's elements one
// instruction takes is free as long as both operands agree, so each lane loads
// consecutive ones, 128 bytes of a row per four lanes and stage, and no weight
// passes through shared memory.  The warps of a CTA take such stages of K in turn,
// the CTAs of a cluster share K when there are few rows, and their fp32 sums are
// added in a fixed order, so a column's sum never depends on timing.
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

constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps;
constexpr int kFewStageWords = 8;       // 32-bit words of a row that a lane loads per stage
constexpr int kFewStageBytes = 4 * 4 * kFewStageWords;      // of a row, by its four lanes

template <typename T>
struct CodeBits;
template <>
struct CodeBits<__nv_bfloat16> {
    static constexpr uint32_t magic = 0x43004300u;      // two times 128
    static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
};
template <>
struct CodeBits<__half> {
    static constexpr uint32_t magic = 0x64006400u;      // two times 1024
    static __device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
};

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
    constexpr int kWords = kCodes ? VEC : 4;                // consecutive words of a lane
    constexpr int kChunks = kFewStageWords / kWords;        // of a stage: 4 lanes x kWords words of a row each
    constexpr int kPerWord = kCodes ? 8 : 2;                // elements of K
    constexpr int kStageK = 4 * kFewStageWords * kPerWord;
    constexpr int kTokens = 8 * NB, kRows = 32, kPitch = kRows + 1;
    __shared__ float sums[kFewWarps][kTokens * kPitch];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int KS = p.k_split, rank = KS > 1 ? (int)cluster_ctarank() : 0;
    const int n0 = (int)(blockIdx.x / KS) * (GATED ? 16 : 32);
    griddep_wait();
    griddep_launch_dependents();

    // this lane's four rows of W: g and g + 8 of both blocks; rows past the last read that one instead and are not stored
    const uint8_t* row_at[4];
    int64_t row_of[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int in = (i & 1) * 8 + g, block = i >> 1;
        const int64_t r = GATED ? (int64_t)block * p.n + min(n0 + in, p.n - 1) : min(n0 + block * 16 + in, p.n - 1);
        row_of[i] = r;
        row_at[i] = static_cast<const uint8_t*>(p.w) + r * p.ldw_bytes + 4 * kWords * t;
    }
    const int stages = (p.k + kStageK - 1) / kStageK;
    const int s_end = (int)((int64_t)stages * (rank + 1) / KS);
    int s = (int)((int64_t)stages * rank / KS) + warp;

    struct Stage {
        uint32_t w[4][kFewStageWords];
        uint32_t factor[kCodes ? 4 : 1][kCodes ? 2 : 1];     // of row i: scale and zero point of the stage's group t (and t + 4)
    };
    auto load = [&](Stage& st, int stage) {
        const int k0 = stage * kStageK;
        const int64_t at = (int64_t)stage * kFewStageBytes;
        if (k0 + kStageK <= p.k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const uint8_t* q = row_at[i] + at + c * (16 * kWords);
                    if constexpr (kWords == 4) {
                        const uint4 v = load_once16(q);
                        st.w[i][4 * c] = v.x;
                        st.w[i][4 * c + 1] = v.y;
                        st.w[i][4 * c + 2] = v.z;
                        st.w[i][4 * c + 3] = v.w;
                    } else if constexpr (kWords == 2) {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
                        st.w[i][2 * c] = v.x;
                        st.w[i][2 * c + 1] = v.y;
                    } else {
                        st.w[i][c] = __ldg(reinterpret_cast<const uint32_t*>(q));
                    }
                }
        } else {
            const int row_bytes = kCodes ? p.k / 2 : 2 * p.k;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int left = row_bytes - (int)at - c * (16 * kWords) - 4 * kWords * t;
                    const uint8_t* q = row_at[i] + at + c * (16 * kWords);
#pragma unroll
                    for (int j = 0; j < kWords; ++j) st.w[i][c * kWords + j] = load_clipped4(q + 4 * j, left - 4 * j);
                }
        }
        if constexpr (kCodes) {
            const int first = k0 / p.group, last = (p.k - 1) / p.group;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < (VEC == 1 ? 2 : 1); ++h) {
                    const int gi = min(first + t + 4 * h, last);
                    const uint32_t sc = __ldg(static_cast<const uint16_t*>(p.scales) + row_of[i] * p.ld_scales + gi);
                    const uint32_t z = p.zeros ? __ldg(p.zeros + row_of[i] * p.ld_zeros + gi) : 8u;
                    st.factor[i][h] = sc | (z << 16);
                }
        }
    };

    float acc[2][NB][4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][nb][i] = 0.f;

    const uint16_t* x_row[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) x_row[nb] = static_cast<const uint16_t*>(p.x) + (int64_t)min(nb * 8 + g, p.tokens - 1) * p.ldx;
    // eight elements of this lane's token at k, zeros past K and for tokens that do not exist
    auto load_x = [&](int nb, int k, bool whole) {
        if (nb * 8 + g >= p.tokens) return make_uint4(0u, 0u, 0u, 0u);
        return whole ? __ldg(reinterpret_cast<const uint4*>(x_row[nb] + k)) : load_clipped16(x_row[nb] + k, 2 * (p.k - k));
    };

    auto multiply = [&](const Stage& st, int stage) {
        const int k0 = stage * kStageK;
        const bool whole = k0 + kStageK <= p.k;
        if constexpr (kCodes) {
            const int first = k0 / p.group;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int kc = k0 + c * 32 * VEC;
                if (kc >= p.k) break;
                const int gi = kc / p.group - first;        // which of the stage's groups
                float part[2][NB][4];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[b][nb][i] = 0.f;
                float scale[4];
                uint32_t zero[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t mine = VEC == 1 && gi >= 4 ? st.factor[i][VEC == 1 ? 1 : 0] : st.factor[i][0];
                    const uint32_t f = __shfl_sync(0xffffffffu, mine, (lane & 28) | (gi & 3));
                    scale[i] = unpack2<T>(f & 0xFFFFu).x;
                    zero[i] = CodeBits<T>::magic + (f >> 16) * 0x10001u;
                }
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    uint32_t xb[NB][4];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint4 q = load_x(nb, kc + 8 * (VEC * t + v), whole);
                        // elements j and j + 4 of a word lie 16 bits apart
                        xb[nb][0] = __byte_perm(q.x, q.z, 0x5410);
                        xb[nb][1] = __byte_perm(q.x, q.z, 0x7632);
                        xb[nb][2] = __byte_perm(q.y, q.w, 0x5410);
                        xb[nb][3] = __byte_perm(q.y, q.w, 0x7632);
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t lo = st.w[2 * b][c * VEC + v], hi = st.w[2 * b + 1][c * VEC + v];
                        uint32_t a[4][2];      // pair j of both rows
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[j][0] = CodeBits<T>::less(((lo >> (4 * j)) & 0x000F000Fu) | CodeBits<T>::magic, zero[2 * b]);
                            a[j][1] = CodeBits<T>::less(((hi >> (4 * j)) & 0x000F000Fu) | CodeBits<T>::magic, zero[2 * b + 1]);
                        }
                        const uint32_t a0[4] = {a[0][0], a[0][1], a[1][0], a[1][1]}, a1[4] = {a[2][0], a[2][1], a[3][0], a[3][1]};
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            mma_16816<T>(part[b][nb], a0, xb[nb][0], xb[nb][1]);
                            mma_16816<T>(part[b][nb], a1, xb[nb][2], xb[nb][3]);
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][nb][i] = fmaf(scale[2 * b + (i >> 1)], part[b][nb][i], acc[b][nb][i]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                uint4 xb[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) xb[nb] = load_x(nb, k0 + 32 * c + 8 * t, whole);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t* lo = st.w[2 * b] + 4 * c;
                    const uint32_t* hi = st.w[2 * b + 1] + 4 * c;
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        mma_16816<T>(acc[b][nb], a0, xb[nb].x, xb[nb].y);
                        mma_16816<T>(acc[b][nb], a1, xb[nb].z, xb[nb].w);
                    }
                }
            }
        }
    };

    Stage st[2];
    if (s < s_end) load(st[0], s);
    while (s < s_end) {
        if (s + kFewWarps < s_end) load(st[1], s + kFewWarps);
        multiply(st[0], s);
        s += kFewWarps;
        if (s >= s_end) break;
        if (s + kFewWarps < s_end) load(st[0], s + kFewWarps);
        multiply(st[1], s);
        s += kFewWarps;
    }

    // ---------------------------------------------------------------- the warps' sums, then the cluster's
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[warp][(nb * 8 + 2 * t + (i & 1)) * kPitch + b * 16 + (i >> 1) * 8 + g] = acc[b][nb][i];
    __syncthreads();
    for (int e = threadIdx.x; e < kTokens * kRows; e += kFewThreads) {
        const int at = (e / kRows) * kPitch + e % kRows;
        float v = sums[0][at];
#pragma unroll
        for (int w = 1; w < kFewWarps; ++w) v += sums[w][at];
        sums[0][at] = v;        // read by this thread alone until the barrier below
    }
    if (KS > 1) cluster_sync(); else __syncthreads();
    constexpr int kOut = GATED ? 16 : 32;       // columns of Y
    const int all = kTokens * kOut, e1 = all * (rank + 1) / KS;
    const uint32_t base = smem_u32(&sums[0][0]);
    auto total = [&](int at) {
        if (KS == 1) return sums[0][at];
        float v = 0.f;
        for (int q = 0; q < KS; ++q) {
            float o;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(map_to_cta(base + 4u * at, (uint32_t)q)));
            v += o;
        }
        return v;
    };
    for (int e = all * rank / KS + threadIdx.x; e < e1; e += kFewThreads) {
        const int token = e / kOut, c = e - token * kOut, n = n0 + c;
        if (token >= p.tokens || n >= p.n) continue;
        float v = total(token * kPitch + c);
        if constexpr (GATED) {
            const float u = total(token * kPitch + 16 + c);
            if (p.gate) {
                static_cast<T*>(p.gate)[(int64_t)token * p.ld_gate_up + n] = (T)v;
                static_cast<T*>(p.up)[(int64_t)token * p.ld_gate_up + n] = (T)u;
            }
            v = activate(p.act, v) * u;
        }
        static_cast<T*>(p.y)[(int64_t)token * p.ldy + n] = (T)v;
    }
    if (KS > 1) cluster_sync_relaxed();     // peers have read this CTA's sums
}

template <typename T, int VEC, int NB, bool GATED>
static cudaError_t launch_few_as(const FewParams& p, cudaStream_t stream) {
    const int64_t tiles = (p.n + (GATED ? 15 : 31)) / (GATED ? 16 : 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.k_split));
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.k_split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.k_split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, few_tokens_kernel<T, VEC, NB, GATED>, p);
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
