// qk_norm_rope.cu -- RMS norm of every query and key head with its rotary
// position in one pass (include/serving.h), forward with an optional append to
// a paged key-value cache, and backward.
//
// A head row of head_dim 16-bit elements is held by 8, 16 or 32 neighbouring
// lanes, eight elements (one 16-byte load) each: a row is read once, its sum
// of squares is reduced by shuffles, and it is written once.  The kernels are
// bound by memory; what competes with it is the instruction count, so a lane
// group takes several rows of one kind (queries, keys or values) of one token
// and prepares their common factors once, and fp32 arithmetic goes two values
// to an instruction.  GB300, heads of 128, 32 of queries and 8 of keys: 16384
// tokens forward with the cache append 69.9 us, 411 MB, 5.9 TB/s, 87% of a plain
// copy's rate; 8192 tokens backward 51.7 us, 256 MB, 4.9 TB/s; 16 tokens forward
// 3.0 us, which is a launch.
//
// With the pairs' rotation y_a' = y_a c - y_b s, y_b' = y_a s + y_b c and
// y = x r w, every element e with partner e' is
//   y_e = r (x_e (w_e c_e) + x_e' (w_e' s_e)),
// s_e = -s for the first element of a pair and +s for the second: the two
// bracketed factors depend on the token and the kind only, and the partners
// are exchanged as loaded, two 16-bit elements to a register.
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
    // Either layout, any even rot: through shared memory.  Bound by its instructions, not by memory (spills of 96 bytes stored,
    // 244 loaded a thread forward): 16384 tokens, 24 of 128 elements rotated as halves, 84.7 us, 20 as neighbours 97.4, where
    // the whole head takes 69.9; 8192 tokens backward, 24 of 128, 71.2 and 51.7.
    kPairsAny = 2
};

enum RowKind { kQueries = 0, kKeys = 1, kValues = 2 };

struct RopeParams {
    qk_norm_rope_args_t a;
    qk_norm_rope_grads_t g;
    int32_t rows_per_group;     // head rows of one token a lane group takes
    uint32_t q_groups, k_groups;    // lane groups per token for queries; for keys (and for values, with a cache)
    uint32_t q_blocks, k_blocks;    // blocks [0, q_blocks) take queries, the next k_blocks keys, the rest values
    float* partials;            // backward: [block][kMaxHeadDim]
};

__device__ __forceinline__ uint4 load_row16(const void* p) {
    return __ldcs(static_cast<const uint4*>(p));
}

// A token's factors for this lane's eight elements: own[i] = w_e c_e, other[i] = w_e' s_e (sign +1: forward; -1: the turn
// back).  `weight` NULL: ones.  Elements that are not rotated: own = w_e, other = 0 (and their partners are taken as 0).
template <typename T, int PAIRS>
__device__ __forceinline__ void load_factors(const qk_norm_rope_args_t& a, const T* weight, int token, int e0, bool act, bool live,
                                             float sign, float (&own)[8], float (&other)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        own[i] = 1.f;
        other[i] = 0.f;
    }
    if (live) {
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
            own[0] = c0.x; own[1] = c0.y; own[2] = c0.z; own[3] = c0.w;
            own[4] = c1.x; own[5] = c1.y; own[6] = c1.z; own[7] = c1.w;
            other[0] = sg * s0.x; other[1] = sg * s0.y; other[2] = sg * s0.z; other[3] = sg * s0.w;
            other[4] = sg * s1.x; other[5] = sg * s1.y; other[6] = sg * s1.z; other[7] = sg * s1.w;
        } else if constexpr (PAIRS == kPairsNeighbours) {
            const float4 cc = *reinterpret_cast<const float4*>(row + e0 / 2);
            const float4 ss = *reinterpret_cast<const float4*>(row + half + e0 / 2);
            own[0] = own[1] = cc.x; own[2] = own[3] = cc.y; own[4] = own[5] = cc.z; own[6] = own[7] = cc.w;
            other[0] = -sign * ss.x; other[1] = sign * ss.x; other[2] = -sign * ss.y; other[3] = sign * ss.y;
            other[4] = -sign * ss.z; other[5] = sign * ss.z; other[6] = -sign * ss.w; other[7] = sign * ss.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                if (e >= a.rot_dim) continue;
                const int at = a.interleaved ? e / 2 : (e < half ? e : e - half);
                const bool second = a.interleaved ? (e & 1) : e >= half;
                own[i] = row[at];
                other[i] = second ? sign * row[half + at] : -sign * row[half + at];
            }
        }
    }
    if (weight == nullptr || !act) return;
    float w[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(weight + e0), w);
    if (live) {
        if constexpr (PAIRS == kPairsHalves) {
            float v[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(weight + (e0 < a.rot_dim / 2 ? e0 + a.rot_dim / 2 : e0 - a.rot_dim / 2)), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] *= v[i];
        } else if constexpr (PAIRS == kPairsNeighbours) {
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] *= w[i ^ 1];
        } else {
            const int half = a.rot_dim / 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                if (e >= a.rot_dim) continue;
                other[i] *= (float)weight[a.interleaved ? (e ^ 1) : (e < half ? e + half : e - half)];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i] *= w[i];
}

// The partners of x[0..7] (packed in `raw`).  `mate`: kPairsHalves, the lane that holds them; `row`: kPairsAny, this lane
// group's shared row.  Called by every lane of the warp.
template <typename T, int PAIRS>
__device__ __forceinline__ void partners(const qk_norm_rope_args_t& a, int e0, bool live, int mate, float* row, const uint4& raw,
                                         const Pair (&x)[4], Pair (&z)[4]) {
    if constexpr (PAIRS == kPairsHalves) {
        uint4 r;
        r.x = __shfl_sync(0xffffffffu, raw.x, mate);
        r.y = __shfl_sync(0xffffffffu, raw.y, mate);
        r.z = __shfl_sync(0xffffffffu, raw.z, mate);
        r.w = __shfl_sync(0xffffffffu, raw.w, mate);
        if (!live) r = make_uint4(0, 0, 0, 0);
        unpack8<T>(r, z);
    } else if constexpr (PAIRS == kPairsNeighbours) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = halves(x[i]);
            z[i] = live ? pair_of(t.y, t.x) : pair_of(0.f);
        }
    } else {
        const int half = a.rot_dim / 2;
        __syncwarp();
        if (live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(row + e0 + 2 * i) = halves(x[i]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = e0 + 2 * i + j;
                const int at = a.interleaved ? (e ^ 1) : (e < half ? e + half : e - half);
                t[j] = e < a.rot_dim ? row[at] : 0.f;
            }
            z[i] = pair_of(t[0], t[1]);
        }
    }
}

__device__ __forceinline__ void as_pairs(const float (&f)[8], Pair (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair_of(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ float sum_of(Pair a) {
    const float2 t = halves(a);
    return t.x + t.y;
}

template <int LANES, int PAIRS>
struct RowLane {
    int e0;        // this lane's first element
    bool act;      // it holds elements of the row
    bool live;     // ... rotated ones
    int mate;      // kPairsHalves: the lane of the warp with the partners
    __device__ __forceinline__ explicit RowLane(const qk_norm_rope_args_t& a) {
        e0 = (threadIdx.x % LANES) * 8;
        act = e0 < a.head_dim;
        live = act && e0 < a.rot_dim;
        const int step = a.rot_dim / 16;
        mate = (threadIdx.x & 31) + (PAIRS == kPairsHalves && live ? (e0 < a.rot_dim / 2 ? step : -step) : 0);
    }
};

// One kind's rows of the forward pass; a block takes one kind only, so that nothing in the row loop asks for it.
template <typename T, int LANES, int PAIRS, int KIND>
__device__ __forceinline__ void forward_rows(const RopeParams& p, uint32_t block, float* srow) {
    constexpr int kAhead = 4;   // rows whose loads are in flight
    const qk_norm_rope_args_t& a = p.a;
    const RowLane<LANES, PAIRS> me(a);
    const int e0 = me.act ? me.e0 : 0;      // lanes past the row read its start and store nothing
    const uint32_t groups = KIND == kQueries ? p.q_groups : p.k_groups;
    const uint32_t items = (uint32_t)a.tokens * groups;
    const uint32_t item = block * (uint32_t)(kRopeThreads / LANES) + threadIdx.x / LANES;
    const bool valid = item < items;
    const int token = valid ? (int)(item / groups) : 0;
    const int h0 = valid ? (int)(item % groups) * p.rows_per_group : 0;
    const int rows = min(p.rows_per_group, (KIND == kQueries ? a.heads : a.kv_heads) - h0);      // at least one
    const bool stores = valid && me.act;

    const T* src = static_cast<const T*>(KIND == kQueries ? a.q : (KIND == kKeys ? a.k : a.v)) + e0;
    int32_t src_step;
    T* dst = nullptr;
    int32_t dst_step = 0;
    if constexpr (KIND == kQueries) {
        src += token * a.q_token + h0 * a.q_head;
        src_step = (int32_t)a.q_head;
        dst = static_cast<T*>(a.q_out) + token * a.q_out_token + h0 * a.q_out_head + e0;
        dst_step = (int32_t)a.q_out_head;
    } else if constexpr (KIND == kKeys) {
        src += token * a.k_token + h0 * a.k_head;
        src_step = (int32_t)a.k_head;
        if (a.k_out) {
            dst = static_cast<T*>(a.k_out) + token * a.k_out_token + h0 * a.k_out_head + e0;
            dst_step = (int32_t)a.k_out_head;
        }
    } else {
        src += token * a.v_token + h0 * a.v_head;
        src_step = (int32_t)a.v_head;
    }
    // Every lane of a warp runs the same number of batches (the shuffles need them all); rows past a group's last one are
    // its last one again, not stored.  The first batch is on its way while positions, table and slots are looked up.
    uint4 raw[kAhead];
    auto load = [&](int b) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = load_row16(src + (int64_t)min(b + u, rows - 1) * src_step);
    };
    load(0);
    // the cache rows of this token
    const bool fp8 = a.dtype_cache == GEMM_E4M3;
    uint8_t* slot_row = nullptr;
    int32_t slot_step = 0;
    float slot_scale = 1.f;
    if (KIND != kQueries && a.k_cache) {
        const int slot = a.slots[token];
        if (slot >= 0 && slot < a.num_pages * a.page_size) {
            const int page = slot / a.page_size, place = slot % a.page_size;
            const int es = fp8 ? 1 : 2;
            const int64_t at = KIND == kKeys ? page * a.k_page + place * a.k_place + h0 * a.k_chead
                                             : page * a.v_page + place * a.v_place + h0 * a.v_chead;
            slot_row = static_cast<uint8_t*>(KIND == kKeys ? a.k_cache : a.v_cache) + (at + e0) * es;
            slot_step = (int32_t)(KIND == kKeys ? a.k_chead : a.v_chead) * es;
            slot_scale = KIND == kKeys ? a.k_scale : a.v_scale;
        }
    }
    auto append = [&](int r, const Pair (&v)[4]) {
        uint8_t* at = slot_row + (int64_t)r * slot_step;
        if (fp8) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = halves(v[i]);
                y[2 * i] = t.x;
                y[2 * i + 1] = t.y;
            }
            uint2 w;
            w.x = e4m3x4(__fdiv_rn(y[0], slot_scale), __fdiv_rn(y[1], slot_scale), __fdiv_rn(y[2], slot_scale), __fdiv_rn(y[3], slot_scale));
            w.y = e4m3x4(__fdiv_rn(y[4], slot_scale), __fdiv_rn(y[5], slot_scale), __fdiv_rn(y[6], slot_scale), __fdiv_rn(y[7], slot_scale));
            *reinterpret_cast<uint2*>(at) = w;
        } else {
            *reinterpret_cast<uint4*>(at) = round8<T>(v);
        }
    };
    Pair own[4], other[4];
    if constexpr (KIND != kValues) {
        float c[8], s[8];
        load_factors<T, PAIRS>(a, a.norm ? static_cast<const T*>(KIND == kQueries ? a.q_weight : a.k_weight) : nullptr, token, me.e0,
                               me.act, me.live, 1.f, c, s);
        as_pairs(c, own);
        as_pairs(s, other);
    }
    const float inv_d = 1.f / (float)a.head_dim;
    for (int b = 0; b < p.rows_per_group; b += kAhead) {
        if (b) load(b);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = b + u;
            const bool on = stores && r < rows;
            if constexpr (KIND == kValues) {
                if (on && slot_row) {
                    if (fp8) {
                        Pair y[4];
                        unpack8<T>(raw[u], y);
                        append(r, y);
                    } else {
                        *reinterpret_cast<uint4*>(slot_row + (int64_t)r * slot_step) = raw[u];
                    }
                }
            } else {
                Pair x[4], z[4];
                unpack8<T>(raw[u], x);
                float inv = 1.f;
                if (a.norm) {
                    Pair sq = x[0] * x[0];
#pragma unroll
                    for (int i = 1; i < 4; ++i) sq = fma2(x[i], x[i], sq);
                    float sum = sum_of(sq);
                    if (!me.act) sum = 0.f;
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    inv = rsqrtf(fmaf(sum, inv_d, a.eps));
                }
                partners<T, PAIRS>(a, me.e0, me.live, me.mate, srow, raw[u], x, z);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = pair_of(inv) * fma2(z[i], other[i], x[i] * own[i]);
                if (on) {
                    if (KIND == kQueries || dst) *reinterpret_cast<uint4*>(dst + (int64_t)r * dst_step) = round8<T>(x);
                    if (KIND == kKeys && slot_row) append(r, x);
                }
            }
        }
    }
}

template <typename T, int LANES, int PAIRS>
__global__ void __launch_bounds__(kRopeThreads, 4) norm_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float scratch[PAIRS == kPairsAny ? (kRopeThreads / LANES) * LANES * 8 : 1];
    griddep_wait();
    griddep_launch_dependents();
    float* srow = scratch + (PAIRS == kPairsAny ? (threadIdx.x / LANES) * LANES * 8 : 0);
    if (blockIdx.x < p.q_blocks) forward_rows<T, LANES, PAIRS, kQueries>(p, blockIdx.x, srow);
    else if (blockIdx.x < p.q_blocks + p.k_blocks) forward_rows<T, LANES, PAIRS, kKeys>(p, blockIdx.x - p.q_blocks, srow);
    else forward_rows<T, LANES, PAIRS, kValues>(p, blockIdx.x - p.q_blocks - p.k_blocks, srow);
}

// Backward: with g the incoming gradient turned back, n = x r, r = rsqrt(mean x^2 + eps):
//   dweight = sum g n,   dx = r (g w - n mean(g w n)) = r (g w - x k),  k = r^2 mean(g w x).
// The two row sums (x^2 and g w x) are reduced side by side.  A block takes queries or keys only, so that one weight and
// one weight gradient stay in registers while its lane groups walk the tokens; it adds its groups' gradients in a fixed
// order and leaves one partial for weight_grad_kernel.
//
// A lane group's work is a sequence of batches of four rows.  While one batch is computed the next one's x, dy and the
// token's cosines and sines come by asynchronous copies into this thread's own places of shared memory (no barriers): held in
// registers instead, the loads of a batch were waited for before its arithmetic began (8192 tokens: 57 us).  Two blocks to
// an SM: three, with two rows to a batch for their registers, take 77 us, batches of sixteen rows 74.
constexpr int kGradAhead = 4;                            // rows of a batch
constexpr int kGradPieces = 2 * kGradAhead + 4;          // 16-byte pieces of a thread's stage: x, dy, table
constexpr int kGradSmem = 2 * kGradPieces * kRopeThreads * 16;

template <typename T, int LANES, int PAIRS>
__global__ void __launch_bounds__(kRopeThreads, 2) norm_rope_backward_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ __align__(16) uint4 staged[];      // [stage][piece][thread]
    __shared__ __align__(16) float scratch[PAIRS == kPairsAny ? (kRopeThreads / LANES) * LANES * 8 : 1];
    __shared__ __align__(16) float sums[kRopeThreads / 32][LANES * 8];
    griddep_wait();
    griddep_launch_dependents();
    const qk_norm_rope_args_t& a = p.a;
    const qk_norm_rope_grads_t& gr = p.g;
    const RowLane<LANES, PAIRS> me(a);
    const int e0 = me.act ? me.e0 : 0;      // lanes past the row read its start and store nothing
    float* srow = scratch + (PAIRS == kPairsAny ? (threadIdx.x / LANES) * LANES * 8 : 0);
    const bool is_q = blockIdx.x < p.q_blocks;
    const uint32_t block = is_q ? blockIdx.x : blockIdx.x - p.q_blocks, blocks = is_q ? p.q_blocks : gridDim.x - p.q_blocks;
    const uint32_t groups = is_q ? p.q_groups : p.k_groups;
    const uint32_t items = (uint32_t)a.tokens * groups;
    const int heads = is_q ? a.heads : a.kv_heads;
    const T* x_base = static_cast<const T*>(is_q ? a.q : a.k) + e0;
    const T* g_base = static_cast<const T*>(is_q ? gr.dq_out : gr.dk_out) + e0;
    T* d_base = static_cast<T*>(is_q ? gr.dq : gr.dk) + e0;
    const int64_t x_token = is_q ? a.q_token : a.k_token, x_head = is_q ? a.q_head : a.k_head;
    const int64_t g_token = is_q ? gr.dq_out_token : gr.dk_out_token, g_head = is_q ? gr.dq_out_head : gr.dk_out_head;
    const int64_t d_token = is_q ? gr.dq_token : gr.dk_token, d_head = is_q ? gr.dq_head : gr.dk_head;
    const int32_t x_step = (int32_t)x_head, g_step = (int32_t)g_head, d_step = (int32_t)d_head;
    const T* weight = a.norm ? static_cast<const T*>(is_q ? a.q_weight : a.k_weight) : nullptr;
    Pair w[4], dw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = pair_of(1.f);
        dw[i] = pair_of(0.f);
    }
    if (weight && me.act) unpack8<T>(*reinterpret_cast<const uint4*>(weight + e0), w);
    const float inv_d = 1.f / (float)a.head_dim;

    const uint32_t step = blocks * (uint32_t)(kRopeThreads / LANES);
    const uint32_t warp_first = block * (uint32_t)(kRopeThreads / LANES) + (threadIdx.x & ~31) / LANES;
    // A place in this lane group's sequence of batches.  `base`, the warp's first group's item, is the same in the whole
    // warp (its first group has the most items), so every lane runs the same number of batches.
    struct Place {
        uint32_t base;
        int batch, token, group, h0, rows;
        bool valid;
    };
    // an item's rows; the first rows of the list stand in for items that do not exist
    auto enter = [&](Place& at) {
        at.valid = at.base + (threadIdx.x & 31) / LANES < items;
        if (!at.valid) at.token = at.group = 0;
        at.h0 = at.group * p.rows_per_group;
        at.rows = min(p.rows_per_group, heads - at.h0);       // at least one
        at.batch = 0;
    };
    const int token_step = (int)(step / groups), group_step = (int)(step % groups);
    auto advance = [&](Place& at) {
        at.batch += kGradAhead;
        if (at.batch < p.rows_per_group) return;
        at.base += step;
        at.token += token_step;
        at.group += group_step;
        if (at.group >= (int)groups) {
            at.group -= (int)groups;
            ++at.token;
        }
        if (at.base < items) enter(at);
    };
    const uint32_t place0 = smem_u32(staged) + threadIdx.x * 16u;
    auto piece = [&](int stage, int i) { return place0 + (uint32_t)(stage * kGradPieces + i) * (kRopeThreads * 16u); };
    const int half = a.rot_dim / 2;
    int position = 0;                    // of the token that is copied next; fetched a batch ahead
    auto fetch_position = [&](const Place& at) {
        if (PAIRS != kPairsAny && me.live && at.base < items && at.batch == 0)
            position = min(max(a.positions[at.token], 0), a.table_rows - 1);
    };
    auto copy = [&](const Place& at, int stage) {
        if (at.base < items) {
            const T* xs = x_base + at.token * x_token + at.h0 * x_head;
            const T* gs = g_base + at.token * g_token + at.h0 * g_head;
            // rows past the group's last one are its last one again, neither stored nor summed
#pragma unroll
            for (int u = 0; u < kGradAhead; ++u) {
                const int r = min(at.batch + u, at.rows - 1);
                cp_async_16(piece(stage, 2 * u), xs + (int64_t)r * x_step);
                cp_async_16(piece(stage, 2 * u + 1), gs + (int64_t)r * g_step);
            }
            if (PAIRS != kPairsAny && me.live && at.batch == 0) {
                const float* row = a.table + (size_t)position * a.rot_dim;
                if constexpr (PAIRS == kPairsHalves) {
                    const int i0 = me.e0 >= half ? me.e0 - half : me.e0;
                    cp_async_16(piece(stage, 2 * kGradAhead), row + i0);
                    cp_async_16(piece(stage, 2 * kGradAhead + 1), row + i0 + 4);
                    cp_async_16(piece(stage, 2 * kGradAhead + 2), row + half + i0);
                    cp_async_16(piece(stage, 2 * kGradAhead + 3), row + half + i0 + 4);
                } else {
                    cp_async_16(piece(stage, 2 * kGradAhead), row + me.e0 / 2);
                    cp_async_16(piece(stage, 2 * kGradAhead + 1), row + half + me.e0 / 2);
                }
            }
        }
        cp_async_commit();
    };

    Place now, ahead;
    now.base = warp_first;
    now.token = now.group = 0;
    if (groups) {
        const uint32_t item = warp_first + (threadIdx.x & 31) / LANES;
        now.token = (int)(item / groups);
        now.group = (int)(item % groups);
    }
    if (now.base < items) enter(now);
    ahead = now;
    fetch_position(ahead);
    copy(ahead, 0);
    if (ahead.base < items) advance(ahead);
    fetch_position(ahead);
    int stage = 0;
    Pair own[4], other[4];
    while (now.base < items) {
        copy(ahead, stage ^ 1);
        const Place after = ahead;
        if (ahead.base < items) advance(ahead);
        fetch_position(ahead);
        cp_async_wait<1>();
        auto staged_piece = [&](int i) { return staged[(stage * kGradPieces + i) * kRopeThreads + threadIdx.x]; };
        if (now.batch == 0) {
            // the turn back: the sines' signs are the forward's negated
            if constexpr (PAIRS == kPairsAny) {
                float c[8], t[8];
                load_factors<T, PAIRS>(a, nullptr, now.token, me.e0, me.act, me.live, -1.f, c, t);
                as_pairs(c, own);
                as_pairs(t, other);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    own[i] = pair_of(1.f);
                    other[i] = pair_of(0.f);
                }
                if (me.live) {
                    if constexpr (PAIRS == kPairsHalves) {
                        const uint4 c[2] = {staged_piece(2 * kGradAhead), staged_piece(2 * kGradAhead + 1)};
                        const uint4 t[2] = {staged_piece(2 * kGradAhead + 2), staged_piece(2 * kGradAhead + 3)};
                        const Pair sg = pair_of(me.e0 >= half ? -1.f : 1.f);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            own[2 * i] = pair_of(__uint_as_float(c[i].x), __uint_as_float(c[i].y));
                            own[2 * i + 1] = pair_of(__uint_as_float(c[i].z), __uint_as_float(c[i].w));
                            other[2 * i] = sg * pair_of(__uint_as_float(t[i].x), __uint_as_float(t[i].y));
                            other[2 * i + 1] = sg * pair_of(__uint_as_float(t[i].z), __uint_as_float(t[i].w));
                        }
                    } else {
                        const uint4 c = staged_piece(2 * kGradAhead), t = staged_piece(2 * kGradAhead + 1);
                        const uint32_t cw[4] = {c.x, c.y, c.z, c.w}, tw[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            own[i] = pair_of(__uint_as_float(cw[i]));
                            other[i] = pair_of(__uint_as_float(tw[i]), -__uint_as_float(tw[i]));
                        }
                    }
                }
            }
        }
        T* ds = d_base + now.token * d_token + now.h0 * d_head;
        const bool stores = now.valid && me.act;
        // kSide rows side by side: their chains of shuffles overlap
        constexpr int kSide = 2;
#pragma unroll
        for (int u0 = 0; u0 < kGradAhead; u0 += kSide) {
            Pair g[kSide][4];
#pragma unroll
            for (int v = 0; v < kSide; ++v) {
                const uint4 rg = staged_piece(2 * (u0 + v) + 1);
                Pair z[4];
                unpack8<T>(rg, g[v]);
                partners<T, PAIRS>(a, me.e0, me.live, me.mate, srow, rg, g[v], z);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[v][i] = fma2(z[i], other[i], g[v][i] * own[i]);
            }
            if (a.norm) {
                Pair x[kSide][4];
                float sq[kSide], dot[kSide];
#pragma unroll
                for (int v = 0; v < kSide; ++v) {
                    unpack8<T>(staged_piece(2 * (u0 + v)), x[v]);
                    Pair squares = x[v][0] * x[v][0], products = (g[v][0] * w[0]) * x[v][0];
#pragma unroll
                    for (int i = 1; i < 4; ++i) {
                        squares = fma2(x[v][i], x[v][i], squares);
                        products = fma2(g[v][i] * w[i], x[v][i], products);
                    }
                    sq[v] = me.act ? sum_of(squares) : 0.f;
                    dot[v] = me.act ? sum_of(products) : 0.f;
                }
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int v = 0; v < kSide; ++v) {
                        sq[v] += __shfl_xor_sync(0xffffffffu, sq[v], o);
                        dot[v] += __shfl_xor_sync(0xffffffffu, dot[v], o);
                    }
#pragma unroll
                for (int v = 0; v < kSide; ++v) {
                    const bool on = stores && now.batch + u0 + v < now.rows;
                    const float inv = rsqrtf(fmaf(sq[v], inv_d, a.eps));
                    const Pair r = pair_of(inv), k = pair_of(-inv * inv * dot[v] * inv_d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (on) dw[i] = fma2(g[v][i] * r, x[v][i], dw[i]);
                        g[v][i] = r * fma2(x[v][i], k, g[v][i] * w[i]);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < kSide; ++v)
                if (stores && now.batch + u0 + v < now.rows)
                    *reinterpret_cast<uint4*>(ds + (int64_t)(now.batch + u0 + v) * d_step) = round8<T>(g[v]);
        }
        now = after;
        stage ^= 1;
    }
    cp_async_wait<0>();
    if (!(is_q ? gr.dq_weight : gr.dk_weight)) return;
    // groups of a warp, then warps of the block, in a fixed order
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 v = halves(dw[i]);
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if ((threadIdx.x & 31) < LANES) *reinterpret_cast<float2*>(&sums[threadIdx.x / 32][me.e0 + 2 * i]) = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < LANES * 8; e += kRopeThreads) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kRopeThreads / 32; ++i) v += sums[i][e];
        p.partials[(size_t)blockIdx.x * kMaxHeadDim + e] = v;
    }
}

// dq_weight / dk_weight = the partials of the blocks of queries / keys, added in a fixed order: 32 columns per block of
// this kernel, 32 strips of partials.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* partials, int q_blocks, int blocks, int head_dim,
                                                           float* dq_weight, float* dk_weight) {
    __shared__ float strip[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int col = threadIdx.x & 31, s = threadIdx.x >> 5;
    const bool keys = blockIdx.y == 1;
    float* out = keys ? dk_weight : dq_weight;
    const int e = blockIdx.x * 32 + col;
    float v = 0.f;
    if (out && e < head_dim) {
        const int end = keys ? blocks : q_blocks;
        for (int b = (keys ? q_blocks : 0) + s; b < end; b += 32 * 8) {
            float x[8];      // eight loads on the way at once
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = b + 32 * u < end ? partials[(size_t)(b + 32 * u) * kMaxHeadDim + e] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += x[u];
        }
    }
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

constexpr int64_t kWorkspaceBytes = (int64_t)kBackwardMaxBlocks * kMaxHeadDim * sizeof(float);

// Strides between heads are held in 32 bits (those between tokens and pages in 64).
bool small_steps(std::initializer_list<int64_t> steps) {
    for (int64_t v : steps)
        if (v < -(int64_t(1) << 29) || v > (int64_t(1) << 29)) return false;
    return true;
}

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
    if (!small_steps({a.q_head, a.k_head})) return GEMM_ERR_UNSUPPORTED;
    if (!forward) return GEMM_OK;
    if (!small_steps({a.q_out_head, a.k_out_head, a.v_head, a.k_chead, a.v_chead})) return GEMM_ERR_UNSUPPORTED;
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

// Cut the rows of every token into lane groups of at most `per_group` rows of one kind.
void cut_rows(RopeParams& p, int64_t per_group) {
    const int64_t most = std::max(p.a.heads, p.a.kv_heads);
    per_group = std::min<int64_t>(std::max<int64_t>(per_group, 1), most);
    for (;;) {
        p.rows_per_group = (int32_t)per_group;
        p.q_groups = (uint32_t)((p.a.heads + per_group - 1) / per_group);
        p.k_groups = (uint32_t)((p.a.kv_heads + per_group - 1) / per_group);
        // numbers of items stay below 2^31
        if ((int64_t)p.a.tokens * std::max(p.q_groups, p.k_groups) <= INT32_MAX - kRopeThreads || per_group >= most) break;
        per_group *= 2;
    }
}

struct LaunchForward {
    RopeParams& p;
    cudaStream_t stream;
    int sms;
    template <typename T, int LANES, int PAIRS>
    cudaError_t operator()() {
        // As few rows per lane group as fit the device at once (four blocks to an SM), eight at most: a group's time is
        // mostly latency up to there.
        const bool values = p.a.k_cache != nullptr;
        const int64_t total = (int64_t)p.a.tokens * (p.a.heads + p.a.kv_heads * (values ? 2 : 1));
        const int64_t resident = (int64_t)sms * 4 * kRopeThreads / LANES, want = (total + resident - 1) / resident;
        cut_rows(p, want <= 1 ? 1 : (want <= 2 ? 2 : (want <= 4 ? 4 : 8)));
        constexpr int64_t kPerBlock = kRopeThreads / LANES;
        const int64_t q = ((int64_t)p.a.tokens * p.q_groups + kPerBlock - 1) / kPerBlock, k = ((int64_t)p.a.tokens * p.k_groups + kPerBlock - 1) / kPerBlock;
        const int64_t blocks = q + k * (values ? 2 : 1);
        p.q_blocks = (uint32_t)q;
        p.k_blocks = (uint32_t)k;
        return launch_dependent(norm_rope_kernel<T, LANES, PAIRS>, dim3((unsigned)blocks), dim3(kRopeThreads), 0, stream, p);
    }
};

struct LaunchBackward {
    RopeParams& p;
    cudaStream_t stream;
    int sms;
    template <typename T, int LANES, int PAIRS>
    cudaError_t operator()() {
        const int64_t total = (int64_t)p.a.tokens * (p.a.heads + p.a.kv_heads);
        const int64_t resident = (int64_t)sms * 2 * kRopeThreads / LANES, want = (total + resident - 1) / resident;
        cut_rows(p, want <= 1 ? 1 : (want <= 2 ? 2 : (want <= 16 ? 4 : 8)));
        // blocks in proportion to the rows, two to an SM (what their registers allow) at most
        constexpr int64_t kPerBlock = kRopeThreads / LANES;
        const int64_t most = std::min<int64_t>(2 * (int64_t)sms, kBackwardMaxBlocks);
        const int64_t q_items = (int64_t)p.a.tokens * p.q_groups, k_items = (int64_t)p.a.tokens * p.k_groups;
        int64_t q = (q_items + kPerBlock - 1) / kPerBlock, k = (k_items + kPerBlock - 1) / kPerBlock;
        if (q + k > most) {
            const int64_t share = most * p.a.heads / (p.a.heads + p.a.kv_heads);
            q = std::min(q, q == 0 ? 0 : std::min(std::max<int64_t>(share, 1), most - (k ? 1 : 0)));
            k = std::min(k, most - q);
        }
        p.q_blocks = (uint32_t)q;
        const bool weights = p.g.dq_weight || p.g.dk_weight;
        p.partials = static_cast<float*>(p.g.workspace);
        static std::atomic<int> smem_set[kMaxDevices];
        auto kern = norm_rope_backward_kernel<T, LANES, PAIRS>;
        cudaError_t e = ensure_smem_limit(kern, kGradSmem, smem_set);
        if (e != cudaSuccess) return e;
        e = launch_dependent(kern, dim3((unsigned)(q + k)), dim3(kRopeThreads), kGradSmem, stream, p);
        if (e != cudaSuccess || !weights) return e;
        return launch_dependent(weight_grad_kernel, dim3((unsigned)((p.a.head_dim + 31) / 32), 2), dim3(1024), 0, stream,
                                (const float*)p.partials, (int)q, (int)(q + k), (int)p.a.head_dim, p.g.dq_weight, p.g.dk_weight);
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
    if (!small_steps({g.dq_out_head, g.dk_out_head, g.dq_head, g.dk_head})) return GEMM_ERR_UNSUPPORTED;
    DeviceFacts dev;
    if ((s = device_facts(&dev)) != GEMM_OK) return s;
    RopeParams p{};
    p.a = *args;
    p.g = g;
    return status_of(with_kernel(p.a, LaunchBackward{p, st, dev.sms}));
}

int64_t qk_norm_rope_backward_workspace(void) { return kWorkspaceBytes; }

}  // extern "C"
