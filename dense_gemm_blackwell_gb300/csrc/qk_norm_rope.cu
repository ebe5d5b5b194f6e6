// qk_norm_rope.cu -- RMS norm of every query and key head with its rotary
// position in one pass (include/serving.h), forward with an optional append to
// a paged key-value cache, and backward.
//
// A head row of head_dim 16-bit elements is held by 8, 16 or 32 neighbouring
// lanes, eight elements (one 16-byte load) each: a row is read once, its sum
// of squares is reduced by shuffles, and it is written once.  A lane group
// takes several rows of one token in turn, so the token's cosines and sines
// (the same for every head) stay in registers.  The kernels are bound by
// memory: four rows' loads (two rows' x and dy in the backward pass) are
// issued before the first is used.
//
// Rotated pairs are y_a' = y_a c - y_b s and y_b' = y_a s + y_b c, written here
// for every element e with partner e' as  y_e' = y_e c + y_e' s_e  with
// s_e = -s for the first element of a pair and +s for the second; the backward
// pass turns the other way (s_e negated).
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "elem.cuh"
#include "serving.h"
#include "serving_host.h"

namespace dgb {

constexpr int kRopeThreads = 256;
constexpr int kBackwardMaxBlocks = 1024;   // partial weight gradients kept in the workspace
constexpr int kMaxHeadDim = 256;

// Where an element's partner is found.
enum RopePairs {
    kPairsHalves = 0,      // elements (i, i + rot/2), rot a multiple of 16: one other lane holds all eight partners
    kPairsNeighbours = 1,  // elements (2i, 2i + 1), rot a multiple of 8
    kPairsAny = 2          // either layout, any even rot: through shared memory
};

struct RopeParams {
    qk_norm_rope_args_t a;
    qk_norm_rope_grads_t g;
    int32_t rows_per_group;   // head rows of one token a lane group takes
    int32_t rows;             // head rows per token (queries, keys and, with a cache, values)
    uint32_t groups;          // lane groups per token
    uint32_t items;           // tokens x groups, below 2^31
    float* partials;          // backward: [block][2][kMaxHeadDim]
};

__device__ __forceinline__ uint4 load_row16(const void* p) {
    return __ldcs(static_cast<const uint4*>(p));
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// This lane's eight cosines and signed sines of a token.  `live`: the lane holds rotated elements.
template <int PAIRS>
__device__ __forceinline__ void load_turn(const qk_norm_rope_args_t& a, int token, int e0, bool live, float sign,
                                          float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
    }
    if (!live) return;
    const int half = a.rot_dim / 2;
    const int pos = min(max(a.positions[token], 0), a.table_rows - 1);
    const float* row = a.table + (size_t)pos * a.rot_dim;
    if constexpr (PAIRS == kPairsHalves) {
        const bool second = e0 >= half;
        const int i0 = second ? e0 - half : e0;
        const float sg = second ? sign : -sign;
        const float4 c0 = *reinterpret_cast<const float4*>(row + i0), c1 = *reinterpret_cast<const float4*>(row + i0 + 4);
        const float4 s0 = *reinterpret_cast<const float4*>(row + half + i0),
                     s1 = *reinterpret_cast<const float4*>(row + half + i0 + 4);
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
        c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = sg * s0.x; s[1] = sg * s0.y; s[2] = sg * s0.z; s[3] = sg * s0.w;
        s[4] = sg * s1.x; s[5] = sg * s1.y; s[6] = sg * s1.z; s[7] = sg * s1.w;
    } else if constexpr (PAIRS == kPairsNeighbours) {
        const float4 cc = *reinterpret_cast<const float4*>(row + e0 / 2);
        const float4 ss = *reinterpret_cast<const float4*>(row + half + e0 / 2);
        c[0] = c[1] = cc.x; c[2] = c[3] = cc.y; c[4] = c[5] = cc.z; c[6] = c[7] = cc.w;
        s[0] = -sign * ss.x; s[1] = sign * ss.x; s[2] = -sign * ss.y; s[3] = sign * ss.y;
        s[4] = -sign * ss.z; s[5] = sign * ss.z; s[6] = -sign * ss.w; s[7] = sign * ss.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            if (e >= a.rot_dim) continue;
            const int at = a.interleaved ? e / 2 : (e < half ? e : e - half);
            const bool second = a.interleaved ? (e & 1) : e >= half;
            c[i] = row[at];
            s[i] = second ? sign * row[half + at] : -sign * row[half + at];
        }
    }
}

// y turned in place.  `mate`: kPairsHalves, the lane that holds the partners; `row`: kPairsAny, this lane group's shared
// row.  Elements past rot_dim keep their bits (a product with s = 0 would turn an infinity into NaN).
template <int PAIRS>
__device__ __forceinline__ void turn(const qk_norm_rope_args_t& a, int e0, bool live, int mate, float* row,
                                     const float (&c)[8], const float (&s)[8], float (&y)[8]) {
    if constexpr (PAIRS == kPairsHalves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = __shfl_sync(0xffffffffu, y[i], mate);
            if (live) y[i] = fmaf(other, s[i], y[i] * c[i]);
        }
    } else if constexpr (PAIRS == kPairsNeighbours) {
        if (live) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float u = y[i], v = y[i + 1];
                y[i] = fmaf(v, s[i], u * c[i]);
                y[i + 1] = fmaf(u, s[i + 1], v * c[i + 1]);
            }
        }
    } else {
        const int half = a.rot_dim / 2;
        __syncwarp();
        if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) row[e0 + i] = y[i];
        }
        __syncwarp();
        if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                if (e >= a.rot_dim) continue;
                const int at = a.interleaved ? (e ^ 1) : (e < half ? e + half : e - half);
                y[i] = fmaf(row[at], s[i], y[i] * c[i]);
            }
        }
        __syncwarp();
    }
}

template <typename T, int LANES, int PAIRS>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kAhead = 4;   // rows whose loads are in flight
    __shared__ float scratch[PAIRS == kPairsAny ? (kRopeThreads / LANES) * LANES * 8 : 1];
    griddep_wait();
    griddep_launch_dependents();
    const qk_norm_rope_args_t& a = p.a;
    const int l = threadIdx.x % LANES;
    const int e0 = l * 8;
    const bool act = e0 < a.head_dim;
    const bool live = act && e0 < a.rot_dim;
    float* srow = scratch + (PAIRS == kPairsAny ? (threadIdx.x / LANES) * LANES * 8 : 0);
    // the lane (of the warp) with the partners of this lane's elements
    const int step = a.rot_dim / 16;
    const int mate = (threadIdx.x & 31) + (PAIRS == kPairsHalves && live ? (e0 < a.rot_dim / 2 ? step : -step) : 0);
    const uint32_t item = blockIdx.x * (uint32_t)(kRopeThreads / LANES) + threadIdx.x / LANES;
    const bool valid = item < p.items;
    const int token = valid ? (int)(item / p.groups) : 0;
    const int r0 = valid ? (int)(item % p.groups) * p.rows_per_group : 0;
    const int r1 = valid ? min(r0 + p.rows_per_group, p.rows) : 0;

    float c[8], s[8];
    load_turn<PAIRS>(a, token, e0, live, 1.f, c, s);
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    const bool has_wq = a.norm && a.q_weight, has_wk = a.norm && a.k_weight;
    if (has_wq && act) wq = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q_weight) + e0);
    if (has_wk && act) wk = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_weight) + e0);
    const float inv_d = 1.f / (float)a.head_dim;
    bool stored = false;        // this token has a cache slot
    int64_t k_at = 0, v_at = 0;
    if (a.k_cache) {
        const int slot = a.slots[token];
        stored = slot >= 0 && slot < a.num_pages * a.page_size;
        const int page = slot / a.page_size, place = slot % a.page_size;
        k_at = page * a.k_page + place * a.k_place;
        v_at = page * a.v_page + place * a.v_place;
    }
    const int H = a.heads, G = a.kv_heads;
    const bool fp8 = a.dtype_cache == GEMM_E4M3;

    auto source = [&](int r) -> const T* {
        if (r < H) return static_cast<const T*>(a.q) + token * a.q_token + r * a.q_head + e0;
        if (r < H + G) return static_cast<const T*>(a.k) + token * a.k_token + (r - H) * a.k_head + e0;
        return static_cast<const T*>(a.v) + token * a.v_token + (r - H - G) * a.v_head + e0;
    };
    auto append = [&](void* cache, int64_t at, float scale, const float (&y)[8]) {
        if (fp8) {
            uint2 w;
            w.x = e4m3x4(__fdiv_rn(y[0], scale), __fdiv_rn(y[1], scale), __fdiv_rn(y[2], scale), __fdiv_rn(y[3], scale));
            w.y = e4m3x4(__fdiv_rn(y[4], scale), __fdiv_rn(y[5], scale), __fdiv_rn(y[6], scale), __fdiv_rn(y[7], scale));
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at + e0) = w;
        } else {
            *reinterpret_cast<uint4*>(static_cast<T*>(cache) + at + e0) = round8<T>(y);
        }
    };
    // every lane of a warp runs the same number of batches (the shuffles need them all)
    for (int b = 0; b < p.rows_per_group; b += kAhead) {
        uint4 raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = r0 + b + u;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (b + u < p.rows_per_group && r < r1 && act) raw[u] = load_row16(source(r));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (b + u >= p.rows_per_group) break;
            const int r = r0 + b + u;
            const bool on = r < r1 && act;
            float y[8];
            unpack8<T>(raw[u], y);
            if (r >= H + G) {
                // values: copied (every lane of the group agrees on r; other groups of the warp may not)
                if (on && stored) append(a.v_cache, v_at + (r - H - G) * a.v_chead, a.v_scale, y);
            }
            const bool is_q = r < H;
            if (a.norm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
                sum = group_sum<LANES>(sum);
                const float inv = rsqrtf(fmaf(sum, inv_d, a.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= inv;
                if (is_q ? has_wq : has_wk) {
                    float w[8];
                    unpack8<T>(is_q ? wq : wk, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] *= w[i];
                }
            }
            turn<PAIRS>(a, e0, live, mate, srow, c, s, y);
            if (!on || r >= H + G) continue;
            if (is_q) {
                *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + token * a.q_out_token + r * a.q_out_head + e0) = round8<T>(y);
            } else {
                const int h = r - H;
                if (a.k_out)
                    *reinterpret_cast<uint4*>(static_cast<T*>(a.k_out) + token * a.k_out_token + h * a.k_out_head + e0) = round8<T>(y);
                if (stored) append(a.k_cache, k_at + h * a.k_chead, a.k_scale, y);
            }
        }
    }
}

// Backward: with g the incoming gradient turned back, n = x r, r = rsqrt(mean x^2 + eps):
//   dweight = sum g n,   dx = r (g w - n mean(g w n)).
// The two row sums (x^2 and g w x; mean(g w n) = r mean(g w x)) are reduced side by side.  A lane group walks items of
// the whole grid and keeps its share of both weight gradients in registers; the block adds its groups' in a fixed order
// and leaves one partial per block for weight_grad_kernel.
template <typename T, int LANES, int PAIRS>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_backward_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kAhead = 2;
    __shared__ float scratch[PAIRS == kPairsAny ? (kRopeThreads / LANES) * LANES * 8 : 1];
    __shared__ float sums[kRopeThreads / 32][2][LANES * 8];
    griddep_wait();
    griddep_launch_dependents();
    const qk_norm_rope_args_t& a = p.a;
    const qk_norm_rope_grads_t& gr = p.g;
    const int l = threadIdx.x % LANES;
    const int e0 = l * 8;
    const bool act = e0 < a.head_dim;
    const bool live = act && e0 < a.rot_dim;
    float* srow = scratch + (PAIRS == kPairsAny ? (threadIdx.x / LANES) * LANES * 8 : 0);
    const int step = a.rot_dim / 16;
    const int mate = (threadIdx.x & 31) + (PAIRS == kPairsHalves && live ? (e0 < a.rot_dim / 2 ? step : -step) : 0);
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    const bool has_wq = a.norm && a.q_weight, has_wk = a.norm && a.k_weight;
    if (has_wq && act) wq = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q_weight) + e0);
    if (has_wk && act) wk = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_weight) + e0);
    const float inv_d = 1.f / (float)a.head_dim;
    const int H = a.heads;
    float dwq[8] = {}, dwk[8] = {};

    const uint32_t groups_grid = gridDim.x * (uint32_t)(kRopeThreads / LANES);
    const uint32_t first = blockIdx.x * (uint32_t)(kRopeThreads / LANES) + threadIdx.x / LANES;
    const uint32_t warp_first = blockIdx.x * (uint32_t)(kRopeThreads / LANES) + (threadIdx.x & ~31) / LANES;
    // warp-uniform trip count: the warp's first group has the most items
    for (uint32_t base = warp_first, item = first; base < p.items; base += groups_grid, item += groups_grid) {
        const bool valid = item < p.items;
        const int token = valid ? (int)(item / p.groups) : 0;
        const int r0 = valid ? (int)(item % p.groups) * p.rows_per_group : 0;
        const int r1 = valid ? min(r0 + p.rows_per_group, p.rows) : 0;
        float c[8], s[8];
        load_turn<PAIRS>(a, token, e0, live, -1.f, c, s);
        for (int b = 0; b < p.rows_per_group; b += kAhead) {
            uint4 rx[kAhead], rg[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int r = r0 + b + u;
                rx[u] = rg[u] = make_uint4(0, 0, 0, 0);
                if (b + u < p.rows_per_group && r < r1 && act) {
                    const bool is_q = r < H;
                    const int h = is_q ? r : r - H;
                    rx[u] = load_row16(is_q ? static_cast<const T*>(a.q) + token * a.q_token + h * a.q_head + e0
                                            : static_cast<const T*>(a.k) + token * a.k_token + h * a.k_head + e0);
                    rg[u] = load_row16(is_q ? static_cast<const T*>(gr.dq_out) + token * gr.dq_out_token + h * gr.dq_out_head + e0
                                            : static_cast<const T*>(gr.dk_out) + token * gr.dk_out_token + h * gr.dk_out_head + e0);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (b + u >= p.rows_per_group) break;
                const int r = r0 + b + u;
                const bool on = r < r1 && act, is_q = r < H;
                const int h = is_q ? r : r - H;
                float x[8], g[8];
                unpack8<T>(rx[u], x);
                unpack8<T>(rg[u], g);
                turn<PAIRS>(a, e0, live, mate, srow, c, s, g);
                if (a.norm) {
                    float gw[8];
                    if (is_q ? has_wq : has_wk) {
                        unpack8<T>(is_q ? wq : wk, gw);
#pragma unroll
                        for (int i = 0; i < 8; ++i) gw[i] *= g[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) gw[i] = g[i];
                    }
                    float sq = 0.f, dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sq = fmaf(x[i], x[i], sq);
                        dot = fmaf(gw[i], x[i], dot);
                    }
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) {
                        sq += __shfl_xor_sync(0xffffffffu, sq, o);
                        dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    }
                    const float inv = rsqrtf(fmaf(sq, inv_d, a.eps));
                    const float k = inv * inv * dot * inv_d;     // r^2 mean(g w x): dx = r (g w - x k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float gn = g[i] * (x[i] * inv);
                        if (on) {
                            if (is_q) dwq[i] += gn;
                            else dwk[i] += gn;
                        }
                        g[i] = inv * fmaf(-x[i], k, gw[i]);
                    }
                }
                if (!on) continue;
                if (is_q) *reinterpret_cast<uint4*>(static_cast<T*>(gr.dq) + token * gr.dq_token + h * gr.dq_head + e0) = round8<T>(g);
                else *reinterpret_cast<uint4*>(static_cast<T*>(gr.dk) + token * gr.dk_token + h * gr.dk_head + e0) = round8<T>(g);
            }
        }
    }
    if (!p.partials) return;
    // groups of a warp, then warps of the block, in a fixed order
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
            dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
        }
        if ((threadIdx.x & 31) < LANES) {
            sums[threadIdx.x / 32][0][e0 + i] = dwq[i];
            sums[threadIdx.x / 32][1][e0 + i] = dwk[i];
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * LANES * 8; t += kRopeThreads) {
        const int which = t / (LANES * 8), e = t % (LANES * 8);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeThreads / 32; ++w) v += sums[w][which][e];
        p.partials[((size_t)blockIdx.x * 2 + which) * kMaxHeadDim + e] = v;
    }
}

// dq_weight / dk_weight = the blocks' partials, added in a fixed order: 32 columns per block, 32 strips of partials.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* partials, int blocks, int head_dim,
                                                           float* dq_weight, float* dk_weight) {
    __shared__ float strip[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int col = threadIdx.x & 31, s = threadIdx.x >> 5;
    const int which = blockIdx.y;
    float* out = which ? dk_weight : dq_weight;
    const int e = blockIdx.x * 32 + col;
    float v = 0.f;
    if (out && e < head_dim)
        for (int b = s; b < blocks; b += 32) v += partials[((size_t)b * 2 + which) * kMaxHeadDim + e];
    strip[s][col] = v;
    __syncthreads();
    if (s == 0 && out && e < head_dim) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += strip[i][col];
        out[e] = t;
    }
}

namespace {

constexpr int64_t kWorkspaceBytes = (int64_t)kBackwardMaxBlocks * 2 * kMaxHeadDim * sizeof(float);

gemm_status_t check_rope(const qk_norm_rope_args_t& a, bool forward) {
    if (a.tokens < 0 || a.heads < 0 || a.kv_heads < 0 || a.head_dim < 1 || a.rot_dim < 0 || a.rot_dim > a.head_dim || (a.rot_dim & 1))
        return GEMM_ERR_INVALID_ARG;
    if (a.dtype != GEMM_BF16 && a.dtype != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    if (a.tokens > (1 << 30) || a.heads > (1 << 16) || a.kv_heads > (1 << 16)) return GEMM_ERR_UNSUPPORTED;
    if (a.head_dim % 8 != 0 || a.head_dim > kMaxHeadDim) return GEMM_ERR_UNSUPPORTED;
    if (a.tokens == 0 || a.heads + a.kv_heads == 0) return GEMM_OK;
    if (a.rot_dim > 0 && (!a.table || !a.positions || a.table_rows < 1)) return GEMM_ERR_INVALID_ARG;
    if ((a.heads > 0 && !a.q) || (a.kv_heads > 0 && !a.k)) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {a.q, a.k, a.q_weight, a.k_weight, a.table})) return GEMM_ERR_ALIGNMENT;
    if (!all_multiples(8, {a.q_token, a.q_head, a.k_token, a.k_head})) return GEMM_ERR_ALIGNMENT;
    if (!forward) return GEMM_OK;
    const bool cache = a.k_cache || a.v_cache;
    if (a.heads > 0 && !a.q_out) return GEMM_ERR_INVALID_ARG;
    if (a.kv_heads > 0 && !a.k_out && !cache) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {a.q_out, a.k_out})) return GEMM_ERR_ALIGNMENT;
    if (!all_multiples(8, {a.q_out_token, a.q_out_head, a.k_out_token, a.k_out_head})) return GEMM_ERR_ALIGNMENT;
    if (cache && a.kv_heads > 0) {
        if (!a.k_cache || !a.v_cache || !a.v || !a.slots || a.page_size < 1 || a.num_pages < 0) return GEMM_ERR_INVALID_ARG;
        if (a.dtype_cache != a.dtype && a.dtype_cache != GEMM_E4M3) return GEMM_ERR_UNSUPPORTED;
        const bool fp8 = a.dtype_cache == GEMM_E4M3;
        if (fp8 && !(a.k_scale > 0.f && a.v_scale > 0.f)) return GEMM_ERR_INVALID_ARG;
        if (!all_aligned(16, {a.v}) || !all_aligned(fp8 ? 8 : 16, {a.k_cache, a.v_cache})) return GEMM_ERR_ALIGNMENT;
        if (!all_multiples(8, {a.v_token, a.v_head, a.k_page, a.k_place, a.k_chead, a.v_page, a.v_place, a.v_chead}))
            return GEMM_ERR_ALIGNMENT;
    }
    return GEMM_OK;
}

int pairs_of(const qk_norm_rope_args_t& a) {
    if (a.rot_dim == 0) return kPairsNeighbours;      // nothing is turned
    if (a.interleaved) return a.rot_dim % 8 == 0 ? kPairsNeighbours : kPairsAny;
    return a.rot_dim % 16 == 0 ? kPairsHalves : kPairsAny;
}

// Calls f.template operator()<T, LANES, PAIRS>().
template <typename T, int LANES, typename F>
cudaError_t with_pairs(int pairs, F&& f) {
    if (pairs == kPairsHalves) return f.template operator()<T, LANES, kPairsHalves>();
    if (pairs == kPairsNeighbours) return f.template operator()<T, LANES, kPairsNeighbours>();
    return f.template operator()<T, LANES, kPairsAny>();
}
template <typename F>
cudaError_t with_kernel(const qk_norm_rope_args_t& a, F&& f) {
    const int pairs = pairs_of(a);
    const int lanes = a.head_dim <= 64 ? 8 : (a.head_dim <= 128 ? 16 : 32);
    if (a.dtype == GEMM_BF16) {
        if (lanes == 8) return with_pairs<__nv_bfloat16, 8>(pairs, f);
        if (lanes == 16) return with_pairs<__nv_bfloat16, 16>(pairs, f);
        return with_pairs<__nv_bfloat16, 32>(pairs, f);
    }
    if (lanes == 8) return with_pairs<__half, 8>(pairs, f);
    if (lanes == 16) return with_pairs<__half, 16>(pairs, f);
    return with_pairs<__half, 32>(pairs, f);
}

// Cut the rows of every token into lane groups of at most `per_group` rows.
void cut_rows(RopeParams& p, int64_t per_group) {
    per_group = std::min<int64_t>(std::max<int64_t>(per_group, 1), p.rows);
    while ((int64_t)p.a.tokens * ((p.rows + per_group - 1) / per_group) > INT32_MAX - kRopeThreads) per_group *= 2;
    p.rows_per_group = (int32_t)per_group;
    p.groups = (uint32_t)((p.rows + per_group - 1) / per_group);
    p.items = (uint32_t)p.a.tokens * p.groups;
}

struct LaunchForward {
    RopeParams& p;
    cudaStream_t stream;
    int sms;
    template <typename T, int LANES, int PAIRS>
    cudaError_t operator()() {
        // Few rows: one row per lane group, so that every SM gets some.  Many: up to twelve rows a group.
        const int64_t total = (int64_t)p.a.tokens * p.rows;
        const int64_t fill = (int64_t)sms * 2048 / LANES;
        const int64_t want = total / std::max<int64_t>(fill, 1);
        cut_rows(p, want < 2 ? 1 : (want < 4 ? 2 : std::min<int64_t>(12, want & ~int64_t(3))));
        const int64_t blocks = ((int64_t)p.items * LANES + kRopeThreads - 1) / kRopeThreads;
        return launch_dependent(norm_rope_kernel<T, LANES, PAIRS>, dim3((unsigned)blocks), dim3(kRopeThreads), 0, stream, p);
    }
};

struct LaunchBackward {
    RopeParams& p;
    cudaStream_t stream;
    int sms;
    template <typename T, int LANES, int PAIRS>
    cudaError_t operator()() {
        const int64_t total = (int64_t)p.a.tokens * p.rows;
        const int64_t fill = (int64_t)sms * 2048 / LANES;
        const int64_t want = total / std::max<int64_t>(fill, 1);
        cut_rows(p, want < 2 ? 1 : (want < 4 ? 2 : 4));
        const int64_t need = ((int64_t)p.items * LANES + kRopeThreads - 1) / kRopeThreads;
        const int blocks = (int)std::min<int64_t>(need, std::min(sms * 4, kBackwardMaxBlocks));
        const bool weights = p.g.dq_weight || p.g.dk_weight;
        p.partials = weights ? static_cast<float*>(p.g.workspace) : nullptr;
        cudaError_t e = launch_dependent(norm_rope_backward_kernel<T, LANES, PAIRS>, dim3((unsigned)blocks), dim3(kRopeThreads), 0,
                                         stream, p);
        if (e != cudaSuccess || !weights) return e;
        return launch_dependent(weight_grad_kernel, dim3((unsigned)((p.a.head_dim + 31) / 32), 2), dim3(1024), 0, stream,
                                (const float*)p.partials, blocks, (int)p.a.head_dim, p.g.dq_weight, p.g.dk_weight);
    }
};

}  // namespace
}  // namespace dgb

using namespace dgb;

extern "C" {

gemm_status_t qk_norm_rope_run(const qk_norm_rope_args_t* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_INVALID_ARG;
    gemm_status_t s = check_rope(*args, true);
    if (s != GEMM_OK) return s;
    if (args->tokens == 0 || args->heads + args->kv_heads == 0) return GEMM_OK;
    DeviceFacts dev;
    if ((s = device_facts(&dev)) != GEMM_OK) return s;
    RopeParams p{};
    p.a = *args;
    if (p.a.kv_heads == 0) p.a.k_cache = p.a.v_cache = nullptr;
    p.rows = p.a.heads + p.a.kv_heads * (p.a.k_cache ? 2 : 1);
    return status_of(with_kernel(p.a, LaunchForward{p, reinterpret_cast<cudaStream_t>(stream), dev.sms}));
}

gemm_status_t qk_norm_rope_backward(const qk_norm_rope_args_t* args, const qk_norm_rope_grads_t* grads,
                                    gemm_stream_t stream) {
    if (!args || !grads) return GEMM_ERR_INVALID_ARG;
    gemm_status_t s = check_rope(*args, false);
    if (s != GEMM_OK) return s;
    const qk_norm_rope_grads_t& g = *grads;
    if ((g.dq_weight && !(args->norm && args->q_weight)) || (g.dk_weight && !(args->norm && args->k_weight)))
        return GEMM_ERR_INVALID_ARG;
    if ((g.dq_weight || g.dk_weight) && (!g.workspace || g.workspace_bytes < kWorkspaceBytes)) return GEMM_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (args->tokens == 0 || args->heads + args->kv_heads == 0) {
        // sums over nothing
        for (float* w : {g.dq_weight, g.dk_weight})
            if (w && cudaMemsetAsync(w, 0, sizeof(float) * (size_t)args->head_dim, st) != cudaSuccess)
                return status_of(cudaGetLastError());
        return GEMM_OK;
    }
    if ((args->heads > 0 && (!g.dq_out || !g.dq)) || (args->kv_heads > 0 && (!g.dk_out || !g.dk))) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {g.dq_out, g.dk_out, g.dq, g.dk, g.workspace})) return GEMM_ERR_ALIGNMENT;
    if (!all_multiples(8, {g.dq_out_token, g.dq_out_head, g.dk_out_token, g.dk_out_head, g.dq_token, g.dq_head, g.dk_token, g.dk_head}))
        return GEMM_ERR_ALIGNMENT;
    DeviceFacts dev;
    if ((s = device_facts(&dev)) != GEMM_OK) return s;
    RopeParams p{};
    p.a = *args;
    p.g = g;
    p.rows = p.a.heads + p.a.kv_heads;
    return status_of(with_kernel(p.a, LaunchBackward{p, st, dev.sms}));
}

int64_t qk_norm_rope_backward_workspace(void) { return kWorkspaceBytes; }

}  // extern "C"
