// add_rms_norm.cu -- the residual's addition and its RMS norm in one pass
// (include/feedforward.h), in 16 bits or as E4M3 codes with the scales that the
// block-scaled products read, and the backward pass.
//
// A row is shared by up to 32 warps, eight elements (16 bytes) a vector, a few
// vectors a thread.  Bound by memory: a block takes row after row, and every
// thread keeps its vectors of the next rows on the way by asynchronous copies into
// places of shared memory that it alone reads, so that no barrier waits for them; a
// row's sums take shuffles and one exchange.  A scale block of 128 (32) columns is
// 16 (4) neighbouring lanes, so its largest magnitude needs shuffles only.  Few
// rows take one vector a thread (the time is latency), many rows more.
//
// Measured, in a graph: 8192 x 8192 bf16 with a residual to codes with fp32 scales 73 us,
// 6.4 TB/s of the 471 MB it needs (the copy rate allows 69; 67 % of the issue slots), to
// 16 bits 91 us, 5.9 TB/s; 8192 x 4096 to 16 bits 47; 1231 x 2893 f16 to MXFP8 codes 7.5
// us; 8 x 4096 2.4 us, a launch (a call from Python takes 13.4 and 4.7 of the last two).
// Rows past 16384 elements take four vectors a thread, which 64 registers do not hold (192
// to 268 bytes spilled): 4096 x 32768 194 us to codes (139 allowed), 193 to 16 bits (158).
// Short rows are bound by
// instructions, which a row's sums and a block's scale cost whatever its length: 32768 x
// 1024 without a residual to MXFP8 31 us where the bytes take 15 (one warp a row, four
// vectors a lane: 27, but 9.2 us instead of 7.6 at 4096 rows with a residual).
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "elem.cuh"
#include "feedforward.h"
#include "serving_host.h"

namespace dgb {

constexpr int kNormMaxHidden = 32768;
constexpr int kNormMaxTokens = 1 << 30;     // rows a few turns ahead are counted in 32 bits
constexpr float kE4M3Max = 448.f;

// Vector v of the weights, zeros past the row's end.
__device__ __forceinline__ uint4 load_weights(const void* weight, int v, int n) {
    const int left = n - 8 * v;
    if (left >= 8) return __ldg(static_cast<const uint4*>(weight) + v);
    if (left <= 0) return make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const uint16_t* e = static_cast<const uint16_t*>(weight) + 8 * v;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) w[i >> 1] |= (uint32_t)e[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector v of a row of n elements to shared memory, zeros past its end (which are not read).
__device__ __forceinline__ void fetch_vector(uint32_t dst, const uint16_t* row, int v, int n) {
    const int bytes = min(16, 2 * (n - 8 * v));
    cp_async_16_zfill(dst, row + (bytes > 0 ? 8 * v : 0), (uint32_t)max(0, bytes));
}

__device__ __forceinline__ void store_vector(void* row, int v, int n, const uint4& q) {
    const int left = n - 8 * v;
    if (left >= 8) {
        static_cast<uint4*>(row)[v] = q;
        return;
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint16_t* e = static_cast<uint16_t*>(row) + 8 * v;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) e[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

__device__ __forceinline__ void store_codes(void* row, int v, int n, uint2 q) {
    const int left = n - 8 * v;
    if (left >= 8) {
        static_cast<uint2*>(row)[v] = q;
        return;
    }
    const uint32_t w[2] = {q.x, q.y};
    uint8_t* e = static_cast<uint8_t*>(row) + 8 * v;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) e[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Exponent byte of the least power of two s >= 2^-126 with top <= 448 s (448 = 1.75 * 2^8); top is not negative.
__device__ __forceinline__ uint32_t e8m0_of(float top) {
    const uint32_t bits = __float_as_uint(top);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(1, min(e, 254));
}

// The word of the scales' tiles that holds the four blocks of vectors v .. v + 15 of a row.
__device__ __forceinline__ uint32_t* scale_word(const add_rms_norm_args_t& a, int row, int v) {
    const int64_t tile = (int64_t)(row / 128) * ((a.hidden + 127) / 128) + v / 16;
    return reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.scales) + tile * 512) + (row % 32) * 4 + row / 32 % 4;
}

struct NormParams {
    add_rms_norm_args_t a;
    int32_t warps;          // of a row
    int32_t rows;           // of a block at a time
    int32_t all_rows;       // tokens, or for tiled scales the tiles' rows
    float over_hidden;      // 1 / hidden
};

constexpr int kOutSame = 0, kOutBlock128 = 1, kOutMx = 2;

// Rows of a thread on the way or in use: two, but for rows past 16384 elements one, as two of theirs may not fit.  (Three and four
// were no faster when they were tried: 8192 x 8192 with a residual to codes 79 and 93 us where two took 79, before other steps
// brought them to 73.)
template <int VPT>
__host__ __device__ constexpr int norm_stages() { return VPT == 4 ? 1 : 2; }

// Instructions count beside the bytes, so the loops over a thread's vectors have no branches: vectors past the row are zeros, and
// only their stores are left out.  n weight = (h weight) r: the product that does not wait for r, and the largest magnitude of a
// scale block, come before the exchange.
template <typename T, int OUT, int VPT, bool RES>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int S = norm_stages<VPT>(), kKinds = RES ? 2 : 1;
    __shared__ float part[2][32];
    extern __shared__ uint4 ring[];         // [S][x, residual][VPT][threads]
    griddep_wait();
    griddep_launch_dependents();
    const add_rms_norm_args_t& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / p.warps, rw = warp - sub * p.warps;
    const int n = a.hidden;
    const int first = rw * 32 + lane, step = p.warps * 32;     // this thread's vectors: first, first + step, ...
    const int stride = gridDim.x * p.rows, threads = blockDim.x;
    int bytes[VPT];
    Pair weight[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        bytes[j] = max(0, min(16, 2 * (n - 8 * v)));
        if (a.weight) {
            unpack8<T>(load_weights(a.weight, v, n), weight[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) weight[j][i] = pair_of(1.f);
        }
    }
    auto fetch = [&](int row, int s) {
        if (row < a.tokens) {
            const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)row * a.ldx;
            const uint16_t* res = RES ? static_cast<const uint16_t*>(a.residual) + (int64_t)row * a.ld_residual : nullptr;
            const uint32_t dst = smem_u32(ring + s * (kKinds * VPT) * threads + threadIdx.x);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int at = bytes[j] > 0 ? 8 * (first + j * step) : 0;
                cp_async_16_zfill(dst + j * threads * 16, x + at, (uint32_t)bytes[j]);
                if constexpr (RES) cp_async_16_zfill(dst + (VPT + j) * threads * 16, res + at, (uint32_t)bytes[j]);
            }
        }
        cp_async_commit();
    };
    int row0 = blockIdx.x * p.rows;
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(row0 + sub + s * stride, s);
    int slot = 0;
    for (int turn = 0; row0 < p.all_rows; row0 += stride, turn ^= 1) {      // the same turns in the whole block
        const int row = row0 + sub;
        const bool live = row < a.tokens;
        Pair y[VPT][4];             // h, then h weight
        float top[VPT];
        Pair squares = pair_of(0.f);
        cp_async_wait<S - 1>();
        const uint4* mine = ring + slot * (kKinds * VPT) * threads + threadIdx.x;
        uint16_t* sum = static_cast<uint16_t*>(a.sum) + (int64_t)row * a.ld_sum;
        if (live) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = first + j * step;
                uint4 q = mine[j * threads];
                unpack8<T>(q, y[j]);
                if constexpr (RES) {
                    Pair r[4];
                    unpack8<T>(mine[(VPT + j) * threads], r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[j][i] = y[j][i] + r[i];
                    // the sum is rounded once, and the norm is that of the rounded sum, which is what the backward pass and
                    // the next layer have
                    q = round8<T>(y[j]);
                    unpack8<T>(q, y[j]);
                }
                if (a.sum && bytes[j] > 0) store_vector(sum, v, n, q);
                top[j] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    squares = fma2(y[j][i], y[j][i], squares);
                    y[j][i] = y[j][i] * weight[j][i];
                    if constexpr (OUT != kOutSame) top[j] = fmaxf(top[j], fmaxf(fabsf(halves(y[j][i]).x), fabsf(halves(y[j][i]).y)));
                }
                if constexpr (OUT != kOutSame) {
#pragma unroll
                    for (int o = 1; o < (OUT == kOutMx ? 4 : 16); o *= 2) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
                }
            }
        }
        float total = warp_sum(halves(squares).x + halves(squares).y);
        if (p.warps > 1) {
            // two turns' places: a warp may be a turn ahead of those that still read
            if (lane == 0) part[turn][warp] = total;
            __syncthreads();
            total = 0.f;
            for (int i = 0; i < p.warps; ++i) total += part[turn][sub * p.warps + i];
        }
        fetch(row + S * stride, slot);
        if (++slot == S) slot = 0;
        if (!live) {
            if (OUT == kOutMx && row < p.all_rows) {
                // the tiles' rows past the matrix: scales of 0
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if ((lane & 15) == 0 && bytes[j] > 0) *scale_word(a, row, first + j * step) = 0u;
            }
            continue;
        }
        const float r = rsqrtf(total * p.over_hidden + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * step;
            const bool in = bytes[j] > 0;
            float inverse;
            if constexpr (OUT == kOutBlock128) {
                const float s = fmaxf(top[j] * r * (1.f / kE4M3Max), 0x1p-100f);
                inverse = __fdividef(1.f, s);
                if (in && (lane & 15) == 0) static_cast<float*>(a.scales)[(int64_t)row * a.ld_scales + v / 16] = s;
            }
            if constexpr (OUT == kOutMx) {
                const uint32_t e = e8m0_of(top[j] * r);
                inverse = __uint_as_float((254u - e) << 23);            // 2^(127 - e); 0 for e = 254, which finite rows do not reach
                // four blocks are one 32-bit word of a tile; blocks past the matrix are 0
                uint32_t word = in ? e : 0u;
                word |= __shfl_down_sync(0xffffffffu, word, 4) << 8;
                word |= __shfl_down_sync(0xffffffffu, word, 8) << 16;
                if (in && (lane & 15) == 0) *scale_word(a, row, v) = word;
            }
            const Pair both = pair_of(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[j][i] = y[j][i] * both;
            if (!in) continue;
            if constexpr (OUT == kOutSame) {
                store_vector(static_cast<uint16_t*>(a.y) + (int64_t)row * a.ldy, v, n, round8<T>(y[j]));
            } else {
                // the scale's reciprocal and its products are rounded in fp32: next to the code's 4 bits nothing
                const Pair scale = pair_of(inverse);
                float2 c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = halves(y[j][i] * scale);
                store_codes(static_cast<uint8_t*>(a.y) + (int64_t)row * a.ldy, v, n,
                            make_uint2(e4m3x4(c[0].x, c[0].y, c[1].x, c[1].y), e4m3x4(c[2].x, c[2].y, c[3].x, c[3].y)));
            }
        }
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------------ backward

constexpr int kNormGradStages = 2;
constexpr int kNormGradBlocks = 608;       // partial weight gradients in the workspace, one a block
constexpr int kNormJoinThreads = 512, kNormJoinColumns = 32, kNormJoinRows = kNormJoinThreads / (kNormJoinColumns / 4);

struct NormGradParams {
    add_rms_norm_grads_t a;
    int32_t warps, rows;
    float over_hidden;
    float* partials;        // [blocks][hidden rounded up to 8], or NULL
};

// 8192 x 4096 bf16 48 us with both kernels, 5.6 TB/s (the bytes take 40): instruction issue (58 % of the slots) at 16 warps an SM, whose
// registers hold the weight gradients; three and four blocks an SM spilled.  The join is 4 of the 48.
// Rows past 16384 elements take eight vectors a thread and spill (192 to 508 bytes): 4096 x 32768 348 us, where the bytes take 158;
// 4096 x 16384, four vectors, 88 of 79.
//
// dh = d_sum + r dy w - h r^3 mean(dy w h): one exchange for both sums of a row.  A thread keeps the same columns in every row
// that its block takes and sums their weight gradients in registers.
template <typename T, int VPT, int S>
__global__ void __launch_bounds__(512) add_rms_norm_backward_kernel(const __grid_constant__ NormGradParams p) {
    __shared__ float2 part[2][16];
    extern __shared__ uint4 ring[];         // [S][h, dy, d_sum][VPT][threads]; at the end the rows' weight gradients
    griddep_wait();
    griddep_launch_dependents();
    const add_rms_norm_grads_t& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / p.warps, rw = warp - sub * p.warps;
    const int n = a.hidden, pitch = (n + 7) & ~7;
    const int first = rw * 32 + lane, step = p.warps * 32;
    const int kinds = a.d_sum ? 3 : 2, stride = gridDim.x * p.rows;
    auto place = [&](int s, int kind, int j) { return ring + ((s * kinds + kind) * VPT + j) * blockDim.x + threadIdx.x; };
    auto fetch = [&](int row, int s) {
        if (row < a.tokens) {
            const uint16_t* h = static_cast<const uint16_t*>(a.h) + (int64_t)row * a.ld_h;
            const uint16_t* g = static_cast<const uint16_t*>(a.dy) + (int64_t)row * a.ld_dy;
            const uint16_t* d = static_cast<const uint16_t*>(a.d_sum) + (a.d_sum ? (int64_t)row * a.ld_d_sum : 0);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = first + j * step;
                fetch_vector(smem_u32(place(s, 0, j)), h, v, n);
                fetch_vector(smem_u32(place(s, 1, j)), g, v, n);
                if (a.d_sum) fetch_vector(smem_u32(place(s, 2, j)), d, v, n);
            }
        }
        cp_async_commit();
    };
    int row0 = blockIdx.x * p.rows;
#pragma unroll
    for (int s = 0; s < S; ++s) fetch(row0 + sub + s * stride, s);
    uint4 weight[VPT];
    Pair dw[VPT][4];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        if (a.weight) weight[j] = load_weights(a.weight, v, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[j][i] = pair_of(0.f);
    }
    int slot = 0, turn = 0;
    for (; row0 < a.tokens; row0 += stride, turn ^= 1) {       // the same turns in the whole block
        const int row = row0 + sub;
        const bool live = row < a.tokens;
        Pair hh = pair_of(0.f), gh = pair_of(0.f);
        cp_async_wait<S - 1>();
        if (live) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                Pair h[4], g[4], w[4];
                unpack8<T>(*place(slot, 0, j), h);
                unpack8<T>(*place(slot, 1, j), g);
                if (a.weight) unpack8<T>(weight[j], w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hh = fma2(h[i], h[i], hh);
                    gh = fma2(a.weight ? g[i] * w[i] : g[i], h[i], gh);
                }
            }
        }
        float2 sums = make_float2(warp_sum(halves(hh).x + halves(hh).y), warp_sum(halves(gh).x + halves(gh).y));
        if (p.warps > 1) {
            // two turns' places: a warp may be a turn ahead of those that still read
            if (lane == 0) part[turn][warp] = sums;
            __syncthreads();
            sums = make_float2(0.f, 0.f);
            for (int i = 0; i < p.warps; ++i) {
                const float2 o = part[turn][sub * p.warps + i];
                sums.x += o.x;
                sums.y += o.y;
            }
        }
        if (live) {
            const float r = rsqrtf(sums.x * p.over_hidden + a.eps);
            const Pair both = pair_of(r), c = pair_of(-(sums.y * p.over_hidden) * r * r * r);       // r^3 alone may overflow
            uint16_t* dh = static_cast<uint16_t*>(a.dh) + (int64_t)row * a.ld_dh;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = first + j * step;
                Pair h[4], g[4], w[4];
                unpack8<T>(*place(slot, 0, j), h);
                unpack8<T>(*place(slot, 1, j), g);
                if (a.weight) unpack8<T>(weight[j], w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    g[i] = g[i] * both;
                    dw[j][i] = fma2(g[i], h[i], dw[j][i]);
                    if (a.weight) g[i] = g[i] * w[i];
                    g[i] = fma2(c, h[i], g[i]);
                }
                if (a.d_sum) {
                    Pair d[4];
                    unpack8<T>(*place(slot, 2, j), d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[i] = g[i] + d[i];
                }
                if (8 * v < n) store_vector(dh, v, n, round8<T>(g));
            }
        }
        fetch(row + S * stride, slot);
        if (++slot == S) slot = 0;
    }
    cp_async_wait<0>();
    if (p.partials == nullptr) return;
    float* to = p.partials + (int64_t)blockIdx.x * pitch;
    float* all = reinterpret_cast<float*>(ring);
    if (p.rows > 1) __syncthreads();        // the ring is free
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        if (8 * v >= n) break;
        float4* q = reinterpret_cast<float4*>(p.rows > 1 ? all + sub * pitch : to) + 2 * v;
        const float2 b0 = halves(dw[j][0]), b1 = halves(dw[j][1]), b2 = halves(dw[j][2]), b3 = halves(dw[j][3]);
        q[0] = make_float4(b0.x, b0.y, b1.x, b1.y);
        q[1] = make_float4(b2.x, b2.y, b3.x, b3.y);
    }
    if (p.rows > 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < pitch; i += blockDim.x) {
            float s = 0.f;
            for (int q = 0; q < p.rows; ++q) s += all[q * pitch + i];
            to[i] = s;
        }
    }
}

// The blocks' partial weight gradients, added in an order that depends on their number alone.
__global__ void __launch_bounds__(kNormJoinThreads) add_rms_norm_join_kernel(const float* partials, int blocks, int n, float* d_weight) {
    __shared__ float4 part[kNormJoinRows][kNormJoinColumns / 4];
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kLanes = kNormJoinColumns / 4;
    const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes;
    const int i = blockIdx.x * kNormJoinColumns + 4 * lane, pitch = (n + 7) & ~7;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& o) { s = make_float4(s.x + o.x, s.y + o.y, s.z + o.z, s.w + o.w); };
    if (i < pitch) {
#pragma unroll 4
        for (int b = slice; b < blocks; b += kNormJoinRows) add(__ldcg(reinterpret_cast<const float4*>(partials + (int64_t)b * pitch + i)));
    }
    part[slice][lane] = s;
    __syncthreads();
    for (int half = kNormJoinRows / 2; half > 0; half /= 2) {
        if (slice < half) {
            add(part[slice + half][lane]);
            part[slice][lane] = s;
        }
        __syncthreads();
    }
    if (slice != 0) return;
    const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (i + q < n) d_weight[i + q] = f[q];
}

// ------------------------------------------------------------------ host

static bool type16(int32_t t) { return t == GEMM_BF16 || t == GEMM_F16; }

// A leading dim: 0 = packed; false where rows would overlap.
static bool settle(int64_t& ld, int64_t least) {
    if (ld == 0) ld = least;
    return ld >= least;
}

// How rows are laid on threads and blocks.
struct NormShape {
    int vpt, warps, rows, stages;
    unsigned threads;
    size_t smem;
    int per_sm;             // blocks that an SM holds
};

constexpr size_t kNormSmem = 224 * 1024;

// `resident`: threads that an SM holds by their registers.
static NormShape norm_shape(int vectors, int vpt, int kinds, int stages, unsigned resident) {
    NormShape s;
    s.vpt = vpt;
    s.warps = (vectors + 32 * vpt - 1) / (32 * vpt);
    s.rows = std::max(1, 4 / s.warps);
    s.threads = (unsigned)(s.rows * s.warps * 32);
    const size_t row = (size_t)s.threads * vpt * kinds * 16;
    s.stages = stages * row <= kNormSmem ? stages : 1;
    s.smem = s.stages * row;
    s.per_sm = (int)std::max<size_t>(1, std::min<size_t>(kNormSmem / (s.smem + 1280), resident / s.threads));
    return s;
}

template <typename T, int OUT, int VPT, bool RES>
static cudaError_t launch_norm(const NormParams& p, const NormShape& s, unsigned blocks, cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    auto kern = add_rms_norm_kernel<T, OUT, VPT, RES>;
    const cudaError_t e = ensure_smem_limit(kern, s.smem, smem_set);
    return e != cudaSuccess ? e : launch_dependent(kern, dim3(blocks), dim3(s.threads), s.smem, stream, p);
}

template <typename T, int OUT>
static cudaError_t launch_norm_vpt(const NormParams& p, const NormShape& s, unsigned blocks, cudaStream_t stream) {
    const bool res = p.a.residual != nullptr;
    switch (s.vpt) {
    case 1: return res ? launch_norm<T, OUT, 1, true>(p, s, blocks, stream) : launch_norm<T, OUT, 1, false>(p, s, blocks, stream);
    case 2: return res ? launch_norm<T, OUT, 2, true>(p, s, blocks, stream) : launch_norm<T, OUT, 2, false>(p, s, blocks, stream);
    default: return res ? launch_norm<T, OUT, 4, true>(p, s, blocks, stream) : launch_norm<T, OUT, 4, false>(p, s, blocks, stream);
    }
}

template <typename T>
static cudaError_t launch_norm_out(const NormParams& p, const NormShape& s, unsigned blocks, cudaStream_t stream) {
    switch (p.a.scale_mode) {
    case GEMM_SCALE_NONE: return launch_norm_vpt<T, kOutSame>(p, s, blocks, stream);
    case GEMM_SCALE_BLOCK_1x128_128x128: return launch_norm_vpt<T, kOutBlock128>(p, s, blocks, stream);
    default: return launch_norm_vpt<T, kOutMx>(p, s, blocks, stream);
    }
}

template <typename T, int VPT>
static cudaError_t launch_grad(const NormGradParams& p, const NormShape& s, unsigned blocks, cudaStream_t stream) {
    static std::atomic<int> smem_one[kMaxDevices], smem_ring[kMaxDevices];
    const bool one = s.stages == 1;
    auto kern = one ? add_rms_norm_backward_kernel<T, VPT, 1> : add_rms_norm_backward_kernel<T, VPT, kNormGradStages>;
    const cudaError_t e = one ? ensure_smem_limit(kern, s.smem, smem_one) : ensure_smem_limit(kern, s.smem, smem_ring);
    return e != cudaSuccess ? e : launch_dependent(kern, dim3(blocks), dim3(s.threads), s.smem, stream, p);
}

template <typename T>
static cudaError_t launch_backward(const NormGradParams& p, const NormShape& s, unsigned blocks, cudaStream_t stream) {
    switch (s.vpt) {
    case 1: return launch_grad<T, 1>(p, s, blocks, stream);
    case 2: return launch_grad<T, 2>(p, s, blocks, stream);
    case 4: return launch_grad<T, 4>(p, s, blocks, stream);
    default: return launch_grad<T, 8>(p, s, blocks, stream);
    }
}

}  // namespace dgb

using namespace dgb;

extern "C" {

gemm_status_t add_rms_norm_run(const add_rms_norm_args_t* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_INVALID_ARG;
    NormParams p{};
    p.a = *args;
    add_rms_norm_args_t& a = p.a;
    if (a.tokens < 0 || a.hidden < 1 || a.reserved0 != 0 || !(a.eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    if (!type16(a.dtype)) return GEMM_ERR_UNSUPPORTED;
    const bool tiled = a.scale_mode == GEMM_SCALE_MX_E8M0_32, blocks128 = a.scale_mode == GEMM_SCALE_BLOCK_1x128_128x128;
    if (a.scale_mode != GEMM_SCALE_NONE && !tiled && !blocks128) return GEMM_ERR_UNSUPPORTED;
    if (a.hidden > kNormMaxHidden || a.tokens > kNormMaxTokens) return GEMM_ERR_UNSUPPORTED;
    const int64_t n = a.hidden;
    if (!settle(a.ldx, n) || !settle(a.ld_residual, n) || !settle(a.ld_sum, n) || !settle(a.ldy, n)) return GEMM_ERR_INVALID_ARG;
    if (blocks128 ? !settle(a.ld_scales, (n + 127) / 128) : a.ld_scales != 0) return GEMM_ERR_INVALID_ARG;
    if (a.tokens == 0) return GEMM_OK;
    if (!a.x || !a.y || a.y == a.sum || (tiled || blocks128) != (a.scales != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {a.x, a.residual, a.weight, a.sum, a.y}) || !all_aligned(tiled ? 16 : 4, {a.scales})) return GEMM_ERR_ALIGNMENT;
    // of a single row no leading dim is used
    if (a.tokens > 1 && (!all_multiples(8, {a.ldx, a.residual ? a.ld_residual : 0, a.sum ? a.ld_sum : 0}) ||
                         a.ldy % (a.scale_mode == GEMM_SCALE_NONE ? 8 : 16) != 0))
        return GEMM_ERR_ALIGNMENT;
    DeviceFacts dev;
    gemm_status_t s = device_facts(&dev);
    if (s != GEMM_OK) return s;
    const int vectors = (int)((n + 7) / 8);
    p.all_rows = tiled ? (a.tokens + 127) / 128 * 128 : a.tokens;
    // one vector a thread while there are few rows, two while a row fits a block so
    int vpt = p.all_rows > 2 * dev.sms && vectors > 32 ? 2 : 1;
    while ((vectors + 32 * vpt - 1) / (32 * vpt) > 32) vpt *= 2;
    const NormShape shape = norm_shape(vectors, vpt, a.residual ? 2 : 1, vpt == 4 ? norm_stages<4>() : norm_stages<2>(), 1024);
    p.warps = shape.warps;
    p.rows = shape.rows;
    p.over_hidden = 1.f / (float)n;
    const unsigned blocks = (unsigned)std::min((p.all_rows + p.rows - 1) / p.rows, dev.sms * shape.per_sm);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(a.dtype == GEMM_BF16 ? launch_norm_out<__nv_bfloat16>(p, shape, blocks, st) : launch_norm_out<__half>(p, shape, blocks, st));
}

int64_t add_rms_norm_backward_workspace(int32_t hidden) {
    return hidden < 1 ? 0 : (int64_t)kNormGradBlocks * ((hidden + 7) / 8 * 8) * (int64_t)sizeof(float);
}

gemm_status_t add_rms_norm_backward(const add_rms_norm_grads_t* args, gemm_stream_t stream) {
    if (!args) return GEMM_ERR_INVALID_ARG;
    NormGradParams p{};
    p.a = *args;
    add_rms_norm_grads_t& a = p.a;
    if (a.tokens < 0 || a.hidden < 1 || !(a.eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
    if (!type16(a.dtype) || a.hidden > kNormMaxHidden || a.tokens > kNormMaxTokens) return GEMM_ERR_UNSUPPORTED;
    const int64_t n = a.hidden;
    if (!settle(a.ld_dy, n) || !settle(a.ld_h, n) || !settle(a.ld_d_sum, n) || !settle(a.ld_dh, n)) return GEMM_ERR_INVALID_ARG;
    if (a.d_weight && (!a.workspace || a.workspace_bytes < add_rms_norm_backward_workspace(a.hidden))) return GEMM_ERR_INVALID_ARG;
    if (!all_aligned(16, {a.dy, a.h, a.weight, a.d_sum, a.dh, a.d_weight, a.workspace})) return GEMM_ERR_ALIGNMENT;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.tokens == 0)      // a sum over nothing
        return a.d_weight ? status_of(cudaMemsetAsync(a.d_weight, 0, sizeof(float) * (size_t)n, st)) : GEMM_OK;
    if (!a.dy || !a.h || !a.dh) return GEMM_ERR_INVALID_ARG;
    if (a.tokens > 1 && !all_multiples(8, {a.ld_dy, a.ld_h, a.d_sum ? a.ld_d_sum : 0, a.ld_dh})) return GEMM_ERR_ALIGNMENT;
    DeviceFacts dev;
    gemm_status_t s = device_facts(&dev);
    if (s != GEMM_OK) return s;
    const int vectors = (int)((n + 7) / 8);
    int vpt = vectors > 32 ? 2 : 1;
    while ((vectors + 32 * vpt - 1) / (32 * vpt) > 16) vpt *= 2;
    NormShape shape = norm_shape(vectors, vpt, a.d_sum ? 3 : 2, kNormGradStages, vpt > 1 ? 512 : 1024);
    p.warps = shape.warps;
    p.rows = shape.rows;
    p.over_hidden = 1.f / (float)n;
    p.partials = a.d_weight ? static_cast<float*>(a.workspace) : nullptr;
    if (p.partials && p.rows > 1) shape.smem = std::max(shape.smem, (size_t)p.rows * (size_t)((n + 7) / 8 * 8) * sizeof(float));
    const int groups = (a.tokens + p.rows - 1) / p.rows;
    const int blocks = std::min({groups, kNormGradBlocks, dev.sms * shape.per_sm});
    cudaError_t e = a.dtype == GEMM_BF16 ? launch_backward<__nv_bfloat16>(p, shape, (unsigned)blocks, st)
                                         : launch_backward<__half>(p, shape, (unsigned)blocks, st);
    if (e == cudaSuccess && a.d_weight)
        e = launch_dependent(add_rms_norm_join_kernel, dim3((unsigned)((n + kNormJoinColumns - 1) / kNormJoinColumns)),
                             dim3(kNormJoinThreads), 0, st, static_cast<const float*>(p.partials), blocks, (int)n, a.d_weight);
    return status_of(e);
}

}  // extern "C"
