// add_rms_norm.cu -- the residual's addition and its RMS norm in one pass
// (include/feedforward.h), in 16 bits or as E4M3 codes with the scales that the
// block-scaled products read, and the backward pass.
//
// A row is held in registers by the threads that share it, eight elements (one
// 16-byte load) a vector: it is read once, its sum of squares is reduced by
// shuffles and one exchange through shared memory, and it is written once.  A
// scale block of 128 (32) columns is 16 (4) neighbouring lanes, so its largest
// magnitude needs shuffles only.  Bound by memory.
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
constexpr float kE4M3Max = 448.f;

// Vector v of a row of n elements, those past its end as zeros.
__device__ __forceinline__ uint4 load_vector(const void* row, int v, int n) {
    const int left = n - 8 * v;
    if (left >= 8) return __ldcs(static_cast<const uint4*>(row) + v);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const uint16_t* e = static_cast<const uint16_t*>(row) + 8 * v;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) w[i >> 1] |= (uint32_t)e[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vector v of the weights, which every row reads again.
__device__ __forceinline__ uint4 load_weights(const void* weight, int v, int n) {
    if (n - 8 * v >= 8) return __ldg(static_cast<const uint4*>(weight) + v);
    return load_vector(weight, v, n);
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

// The sum of `v` over a row's `warps` warps, the same in each of its threads.  `part` [rows][warps] of the block, not in use by
// an earlier call that threads may still read.  Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, int warps, float* part, int row, int warp) {
    v = warp_sum(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[row * warps + warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += part[row * warps + i];
    return s;
}

// Exponent byte of the least power of two s >= 2^-126 with top <= 448 s (448 = 1.75 * 2^8); top is not negative.
__device__ __forceinline__ uint32_t e8m0_of(float top) {
    const uint32_t bits = __float_as_uint(top);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(1, min(e, 254));
}

struct NormParams {
    add_rms_norm_args_t a;
    int32_t warps;          // of a row
    int32_t rows;           // of a block
    int32_t all_rows;       // tokens, or for tiled scales the tiles' rows
    float over_hidden;      // 1 / hidden
};

constexpr int kOutSame = 0, kOutBlock128 = 1, kOutMx = 2;

template <typename T, int OUT, int VPT>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[32];
    griddep_wait();
    griddep_launch_dependents();
    const add_rms_norm_args_t& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / p.warps, rw = warp - sub * p.warps;
    const int n = a.hidden, row = blockIdx.x * p.rows + sub;
    const int first = rw * 32 + lane, step = p.warps * 32;     // this thread's vectors: first, first + step, ...
    const bool live = row < a.tokens;
    uint4 h[VPT], weight[VPT];      // the row as it is kept, 16 bits an element
    float squares = 0.f;
    if (live) {
        const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)row * a.ldx;
        const uint16_t* res = static_cast<const uint16_t*>(a.residual) + (a.residual ? (int64_t)row * a.ld_residual : 0);
        uint16_t* sum = static_cast<uint16_t*>(a.sum) + (a.sum ? (int64_t)row * a.ld_sum : 0);
        uint4 qr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * step;
            if (8 * v >= n) break;
            h[j] = load_vector(x, v, n);
            if (a.residual) qr[j] = load_vector(res, v, n);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * step;
            if (8 * v >= n) break;
            if (a.weight) weight[j] = load_weights(a.weight, v, n);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * step;
            if (8 * v >= n) break;
            float f[8];
            unpack8<T>(h[j], f);
            if (a.residual) {
                float r[8];
                unpack8<T>(qr[j], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += r[i];
                // the sum is rounded once, and the norm is that of the rounded sum, which is what the backward pass and the
                // next layer have
                h[j] = round8<T>(f);
                unpack8<T>(h[j], f);
            }
            if (a.sum) store_vector(sum, v, n, h[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) squares = fmaf(f[i], f[i], squares);
        }
    }
    const float r = rsqrtf(row_sum(squares, p.warps, part, sub, rw) * p.over_hidden + a.eps);
    if (OUT != kOutMx && !live) return;
    if (row >= p.all_rows) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        if (8 * (v - lane) >= n) break;            // whole warps: the lanes' largest magnitudes are exchanged
        const bool in = live && 8 * v < n;
        float y[8];
        if (in) {
            unpack8<T>(h[j], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= r;
            if (a.weight) {
                float w[8];
                unpack8<T>(weight[j], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.f;
        }
        if constexpr (OUT == kOutSame) {
            if (in) store_vector(static_cast<uint16_t*>(a.y) + (int64_t)row * a.ldy, v, n, round8<T>(y));
        } else {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float inverse;
            if constexpr (OUT == kOutBlock128) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                const float s = fmaxf(top / kE4M3Max, 0x1p-100f);
                inverse = 1.f / s;
                if (in && (lane & 15) == 0) static_cast<float*>(a.scales)[(int64_t)row * a.ld_scales + v / 16] = s;
            } else {
                const uint32_t e = e8m0_of(top);
                inverse = __uint_as_float((254u - e) << 23);        // 2^(127 - e); 0 for e = 254, which finite rows do not reach
                // four blocks are one 32-bit word of a tile; blocks past the matrix are 0
                uint32_t word = in ? e : 0u;
                word |= __shfl_down_sync(0xffffffffu, word, 4) << 8;
                word |= __shfl_down_sync(0xffffffffu, word, 8) << 16;
                if ((lane & 15) == 0 && 8 * v < n) {
                    const int64_t tile = (int64_t)(row / 128) * ((n + 127) / 128) + v / 16;
                    reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.scales) + tile * 512)[(row % 32) * 4 + row / 32 % 4] = word;
                }
            }
            if (in) {
                // the scale's reciprocal and its product with y are rounded in fp32: next to the code's 4 bits nothing
                const uint2 q = make_uint2(e4m3x4(y[0] * inverse, y[1] * inverse, y[2] * inverse, y[3] * inverse),
                                           e4m3x4(y[4] * inverse, y[5] * inverse, y[6] * inverse, y[7] * inverse));
                store_codes(static_cast<uint8_t*>(a.y) + (int64_t)row * a.ldy, v, n, q);
            }
        }
    }
}

// ------------------------------------------------------------------ backward

constexpr int kNormGradBlocks = 608;       // partial weight gradients in the workspace, one a block
constexpr int kNormJoinColumns = 32, kNormJoinRows = 16;

struct NormGradParams {
    add_rms_norm_grads_t a;
    int32_t warps, rows;
    float over_hidden;
    float* partials;        // [blocks][hidden rounded up to 8], or NULL
};

// dh = d_sum + r dy w - h r^3 mean(dy w h): one exchange for both sums of a row.  A thread keeps the same columns in every row
// that its block takes and sums their weight gradients, in registers, or for wide rows (SHARED: registers hold the row) in
// shared memory, each thread its own words.
template <typename T, int VPT, bool SHARED>
__global__ void __launch_bounds__(SHARED ? 1024 : 512, SHARED ? 1 : 2)
add_rms_norm_backward_kernel(const __grid_constant__ NormGradParams p) {
    __shared__ float2 part[2][32];
    extern __shared__ float4 sums_smem[];       // [rows of the block][padded hidden], fp32
    griddep_wait();
    griddep_launch_dependents();
    const add_rms_norm_grads_t& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / p.warps, rw = warp - sub * p.warps;
    const int n = a.hidden, pitch = (n + 7) & ~7;
    const int first = rw * 32 + lane, step = p.warps * 32;
    float4* mine = sums_smem + sub * (pitch / 4);
    float dw[SHARED ? 1 : VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        if constexpr (SHARED) {
            if (p.partials && 8 * v < n) mine[2 * v] = mine[2 * v + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
        }
    }
    const int stride = gridDim.x * p.rows;
    int turn = 0;
    for (int row0 = blockIdx.x * p.rows; row0 < a.tokens; row0 += stride, turn ^= 1) {       // the same turns in the whole block
        const int row = row0 + sub;
        const bool live = row < a.tokens;
        uint4 qh[VPT], qg[VPT], qs[SHARED ? 1 : VPT];
        const uint16_t* ds = static_cast<const uint16_t*>(a.d_sum) + (a.d_sum && live ? (int64_t)row * a.ld_d_sum : 0);
        float2 sums = make_float2(0.f, 0.f);
        if (live) {
            const uint16_t* h = static_cast<const uint16_t*>(a.h) + (int64_t)row * a.ld_h;
            const uint16_t* g = static_cast<const uint16_t*>(a.dy) + (int64_t)row * a.ld_dy;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = first + j * step;
                if (8 * v >= n) break;
                qh[j] = load_vector(h, v, n);
                qg[j] = load_vector(g, v, n);
                if constexpr (!SHARED)
                    if (a.d_sum) qs[j] = load_vector(ds, v, n);
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = first + j * step;
                if (8 * v >= n) break;
                float x[8], g8[8];
                unpack8<T>(qh[j], x);
                unpack8<T>(qg[j], g8);
                if (a.weight) {
                    float w[8];
                    unpack8<T>(load_weights(a.weight, v, n), w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) g8[i] *= w[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sums.x = fmaf(x[i], x[i], sums.x);
                    sums.y = fmaf(g8[i], x[i], sums.y);
                }
            }
        }
        sums.x = warp_sum(sums.x);
        sums.y = warp_sum(sums.y);
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
        if (!live) continue;
        const float r = rsqrtf(sums.x * p.over_hidden + a.eps);
        const float c = r * r * r * (sums.y * p.over_hidden);
        uint16_t* dh = static_cast<uint16_t*>(a.dh) + (int64_t)row * a.ld_dh;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * step;
            if (8 * v >= n) break;
            float x[8], g8[8], o[8];
            unpack8<T>(qh[j], x);
            unpack8<T>(qg[j], g8);
#pragma unroll
            for (int i = 0; i < 8; ++i) g8[i] *= r;
            if constexpr (SHARED) {
                if (p.partials) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float4 t = mine[2 * v + q];
                        t.x = fmaf(g8[4 * q], x[4 * q], t.x);
                        t.y = fmaf(g8[4 * q + 1], x[4 * q + 1], t.y);
                        t.z = fmaf(g8[4 * q + 2], x[4 * q + 2], t.z);
                        t.w = fmaf(g8[4 * q + 3], x[4 * q + 3], t.w);
                        mine[2 * v + q] = t;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[j][i] = fmaf(g8[i], x[i], dw[j][i]);
            }
            if (a.weight) {
                float w[8];
                unpack8<T>(load_weights(a.weight, v, n), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) g8[i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(-c, x[i], g8[i]);
            if (a.d_sum) {
                float d[8];
                if constexpr (SHARED) unpack8<T>(load_vector(ds, v, n), d);
                else unpack8<T>(qs[j], d);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += d[i];
            }
            store_vector(dh, v, n, round8<T>(o));
        }
    }
    if (p.partials == nullptr) return;
    float* to = p.partials + (int64_t)blockIdx.x * pitch;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = first + j * step;
        if (8 * v >= n) break;
        float4 lo, hi;
        if constexpr (SHARED) {
            lo = mine[2 * v];
            hi = mine[2 * v + 1];
        } else {
            lo = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            hi = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        }
        float4* q = p.rows > 1 ? mine : reinterpret_cast<float4*>(to);
        q[2 * v] = lo;
        q[2 * v + 1] = hi;
    }
    if (p.rows > 1) {
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(sums_smem);
        for (int i = threadIdx.x; i < pitch; i += blockDim.x) {
            float s = 0.f;
            for (int q = 0; q < p.rows; ++q) s += all[q * pitch + i];
            to[i] = s;
        }
    }
}

// The blocks' partial weight gradients, added in an order that depends on their number alone.
__global__ void __launch_bounds__(kNormJoinColumns* kNormJoinRows) add_rms_norm_join_kernel(const float* partials, int blocks, int n,
                                                                                            float* d_weight) {
    __shared__ float part[kNormJoinRows][kNormJoinColumns + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % kNormJoinColumns, slice = threadIdx.x / kNormJoinColumns;
    const int i = blockIdx.x * kNormJoinColumns + lane, pitch = (n + 7) & ~7;
    float s = 0.f;
    if (i < n)
        for (int b = slice; b < blocks; b += kNormJoinRows) s += partials[(int64_t)b * pitch + i];
    part[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && i < n) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < kNormJoinRows; ++q) s += part[q][lane];
        d_weight[i] = s;
    }
}

// ------------------------------------------------------------------ host

static bool type16(int32_t t) { return t == GEMM_BF16 || t == GEMM_F16; }

// A leading dim: 0 = packed; false where rows would overlap.
static bool settle(int64_t& ld, int64_t least) {
    if (ld == 0) ld = least;
    return ld >= least;
}

template <typename T, int OUT>
static cudaError_t launch_norm(const NormParams& p, int vpt, unsigned blocks, unsigned threads, cudaStream_t stream) {
    switch (vpt) {
    case 1: return launch_dependent(add_rms_norm_kernel<T, OUT, 1>, dim3(blocks), dim3(threads), 0, stream, p);
    case 2: return launch_dependent(add_rms_norm_kernel<T, OUT, 2>, dim3(blocks), dim3(threads), 0, stream, p);
    default: return launch_dependent(add_rms_norm_kernel<T, OUT, 4>, dim3(blocks), dim3(threads), 0, stream, p);
    }
}

template <typename T>
static cudaError_t launch_norm_out(const NormParams& p, int vpt, unsigned blocks, unsigned threads, cudaStream_t stream) {
    switch (p.a.scale_mode) {
    case GEMM_SCALE_NONE: return launch_norm<T, kOutSame>(p, vpt, blocks, threads, stream);
    case GEMM_SCALE_BLOCK_1x128_128x128: return launch_norm<T, kOutBlock128>(p, vpt, blocks, threads, stream);
    default: return launch_norm<T, kOutMx>(p, vpt, blocks, threads, stream);
    }
}

constexpr int kNormGradNarrow = 8192;      // the widest rows whose weight gradients a thread sums in registers

template <typename T>
static cudaError_t launch_backward(const NormGradParams& p, int vpt, unsigned blocks, unsigned threads, size_t smem, cudaStream_t stream) {
    switch (vpt) {
    case 1: return launch_dependent(add_rms_norm_backward_kernel<T, 1, false>, dim3(blocks), dim3(threads), smem, stream, p);
    case 2: return launch_dependent(add_rms_norm_backward_kernel<T, 2, false>, dim3(blocks), dim3(threads), smem, stream, p);
    }
    static std::atomic<int> smem_set[kMaxDevices];
    const cudaError_t e = ensure_smem_limit(add_rms_norm_backward_kernel<T, 4, true>, smem, smem_set);
    return e != cudaSuccess ? e : launch_dependent(add_rms_norm_backward_kernel<T, 4, true>, dim3(blocks), dim3(threads), smem, stream, p);
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
    if (a.hidden > kNormMaxHidden) return GEMM_ERR_UNSUPPORTED;
    const int64_t n = a.hidden;
    if (!settle(a.ldx, n) || !settle(a.ld_residual, n) || !settle(a.ld_sum, n) || !settle(a.ldy, n)) return GEMM_ERR_INVALID_ARG;
    if (blocks128 ? !settle(a.ld_scales, (n + 127) / 128) : a.ld_scales != 0) return GEMM_ERR_INVALID_ARG;
    if (a.tokens == 0) return GEMM_OK;
    if (!a.x || !a.y || (tiled || blocks128) != (a.scales != nullptr)) return GEMM_ERR_INVALID_ARG;
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
    int vpt = 1;
    while (vpt < 4 && (vectors + 32 * vpt - 1) / (32 * vpt) > 32) vpt *= 2;
    p.warps = (vectors + 32 * vpt - 1) / (32 * vpt);
    p.rows = std::max(1, 8 / p.warps);
    p.over_hidden = 1.f / (float)n;
    const unsigned blocks = (unsigned)((p.all_rows + p.rows - 1) / p.rows), threads = (unsigned)(p.rows * p.warps * 32);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(a.dtype == GEMM_BF16 ? launch_norm_out<__nv_bfloat16>(p, vpt, blocks, threads, st)
                                          : launch_norm_out<__half>(p, vpt, blocks, threads, st));
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
    if (!type16(a.dtype) || a.hidden > kNormMaxHidden) return GEMM_ERR_UNSUPPORTED;
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
    const bool wide = n > kNormGradNarrow;
    const int vpt = wide ? 4 : vectors > 128 ? 2 : 1;
    p.warps = (vectors + 32 * vpt - 1) / (32 * vpt);
    p.rows = std::max(1, 8 / p.warps);
    p.over_hidden = 1.f / (float)n;
    p.partials = a.d_weight ? static_cast<float*>(a.workspace) : nullptr;
    const unsigned threads = (unsigned)(p.rows * p.warps * 32);
    const int groups = (a.tokens + p.rows - 1) / p.rows;
    const int blocks = std::min({groups, kNormGradBlocks, dev.sms * (wide ? 1 : threads <= 256 ? 4 : 2)});
    const size_t smem = p.partials && (wide || p.rows > 1) ? (size_t)p.rows * (size_t)((n + 7) / 8 * 8) * sizeof(float) : 0;
    cudaError_t e = a.dtype == GEMM_BF16 ? launch_backward<__nv_bfloat16>(p, vpt, (unsigned)blocks, threads, smem, st)
                                         : launch_backward<__half>(p, vpt, (unsigned)blocks, threads, smem, st);
    if (e == cudaSuccess && a.d_weight)
        e = launch_dependent(add_rms_norm_join_kernel, dim3((unsigned)((n + kNormJoinColumns - 1) / kNormJoinColumns)),
                             dim3(kNormJoinColumns * kNormJoinRows), 0, st, static_cast<const float*>(p.partials), blocks, (int)n, a.d_weight);
    return status_of(e);
}

}  // extern "C"
