/*
 * feedforward.h -- C ABI of the operators of a feed-forward block, next to
 * gemm.h and serving.h and in the same library:
 *
 *   add_rms_norm_*  the residual's addition and its RMS norm in one pass, in 16
 *                   bits or as E4M3 codes with the scales that the products of
 *                   gemm.h read; and the backward pass
 *   gated_*         H = act(X Wg^T) * (X Wu^T): both projections, the activation
 *                   and the product in one kernel; and the backward pass
 *   int4_matmul_*   products of a few tokens with 4-bit weights and group scales,
 *                   alone or as such a gated pair
 *
 * Conventions are serving.h's: every call returns a gemm_status_t and nothing
 * throws across the ABI; the caller owns every buffer and the stream; calls only
 * enqueue work (no allocation, no synchronisation), so they may be captured into
 * a CUDA graph; unsupported requests fail with GEMM_ERR_UNSUPPORTED.  Strides and
 * leading dimensions count elements.  Work goes to the current device; a plan
 * runs on the device it was made on (GEMM_ERR_INVALID_ARG where another one is
 * current), on one stream, from one host thread, at a time.  Outputs must not
 * overlap inputs or one another except where it is said.
 */
#ifndef DENSE_GEMM_BLACKWELL_GB300_FEEDFORWARD_H
#define DENSE_GEMM_BLACKWELL_GB300_FEEDFORWARD_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ residual, RMS norm, output in 8 bits */

/* h = x + residual, rounded to dtype (no residual: h = x);  n = h * rsqrt(mean(h^2) + eps) * weight, fp32 (a NULL weight: ones).
 * scale_mode says what y holds:
 *   GEMM_SCALE_NONE                n in dtype, rounded once
 *   GEMM_SCALE_BLOCK_1x128_128x128 E4M3 codes e4m3(n / s) and fp32 scales s = max(max|n| / 448, 2^-100) of every 128 columns:
 *                                  gemm_run's A and scale_a
 *   GEMM_SCALE_MX_E8M0_32          E4M3 codes and E8M0 scales of every 32 columns in gemm.h's tiles: gemm_run_mx's A and sf_a.
 *                                  s is the least power of two, at least 2^-126, with max|n| <= 448 s.  All bytes of the
 *                                  ceil(tokens/128) x ceil(hidden/128) tiles are written, those past the matrix as 0.
 * Codes are rounded to nearest even and saturate at +-448.  A NaN weight gives the code of NaN in its column, and the block's
 * scale is that of its other values; a NaN in h makes all of its row NaN, whose scales then say nothing.  Infinite h gives NaN at
 * its place and zeros in the rest of the row.  Squares are summed in fp32: rows with |h| past about 1e18 give zeros, and without
 * eps rows whose |h| are all under about 1e-19 lose bits and under 1e-23 are infinite or NaN. */
typedef struct {
    int32_t tokens, hidden;     /* hidden 1..32768; tokens 0 (no-op) .. 2^30 */
    int32_t dtype;              /* GEMM_BF16 or GEMM_F16: x, residual, weight, sum and an unscaled y */
    int32_t scale_mode;
    float eps;
    int32_t reserved0;          /* must be 0 */
    const void* x;              /* x[t * ldx + i]; rows 16-byte aligned, like all rows here (leading dims: multiples of 16 bytes, 0 = packed) */
    const void* residual;       /* or NULL */
    const void* weight;         /* [hidden], 16-byte aligned, or NULL */
    void* sum;                  /* h; NULL = not wanted; may be residual or x itself (same leading dim) */
    void* y;                    /* GEMM_SCALE_NONE: may be x or residual itself (same leading dim) unless that is sum's place */
    void* scales;               /* fp32 [tokens][ld_scales] (4-byte aligned) or the tiles (16-byte aligned); NULL for GEMM_SCALE_NONE */
    int64_t ldx, ld_residual, ld_sum, ldy, ld_scales;   /* ld_scales: 0 = ceil(hidden / 128); 0 for tiles */
} add_rms_norm_args_t;

/* add_rms_norm_run -- enqueue the forward pass.  GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_ALIGNMENT,
 * GEMM_ERR_NO_DEVICE or GEMM_ERR_CUDA. */
gemm_status_t add_rms_norm_run(const add_rms_norm_args_t* args, gemm_stream_t stream);

/* add_rms_norm_backward -- dh = d_sum + r (dy w - u mean(dy w u)) with r = rsqrt(mean(h^2) + eps), u = h r: the gradient of x
 * and of the residual alike; d_weight = sum over tokens of dy u, in a fixed order.  dy is the gradient of n. */
typedef struct {
    int32_t tokens, hidden;     /* as above; tokens 0: d_weight is zeroed */
    int32_t dtype;
    float eps;
    const void* dy;
    const void* h;              /* the forward pass's sum (x itself without a residual) */
    const void* weight;         /* or NULL */
    const void* d_sum;          /* gradient that reaches h along the residual, or NULL */
    void* dh;                   /* may be dy, d_sum or h itself (same leading dim) */
    float* d_weight;            /* [hidden], 16-byte aligned, or NULL (not wanted) */
    void* workspace;            /* add_rms_norm_backward_workspace(hidden) bytes, 16-byte aligned, when d_weight is wanted */
    int64_t workspace_bytes;
    int64_t ld_dy, ld_h, ld_d_sum, ld_dh;
} add_rms_norm_grads_t;
gemm_status_t add_rms_norm_backward(const add_rms_norm_grads_t* args, gemm_stream_t stream);
int64_t add_rms_norm_backward_workspace(int32_t hidden);

/* ------------------------------------------------------------------ a gated pair of projections */

typedef enum { GATED_SILU = 0, GATED_GELU = 1, GATED_GELU_TANH = 2, GATED_NONE = 3 } gated_activation_t;

/* G = X Wg^T, U = X Wu^T, H = act(G) * U; X is tokens x k, W = [Wg; Wu] is 2 features x k, H is tokens x features.
 * silu(g) = g / (1 + e^-g); gelu(g) = g (1 + erf(g / sqrt 2)) / 2; gelu_tanh(g) = g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2.
 * Sums, activation and product are fp32; H, and G and U where they are kept, are rounded once. */
typedef struct {
    int64_t tokens, features, k;    /* features a multiple of 8; tokens 0 = no-op */
    int32_t activation;             /* GATED_SILU, GATED_GELU or GATED_GELU_TANH */
    int32_t dtype;                  /* GEMM_BF16 or GEMM_F16: everything but d_w */
    int32_t gradients;              /* 1: the plan also runs backward passes */
    int32_t dtype_dw;               /* dtype or GEMM_F32 */
    int64_t ldx, ldw, ldh;          /* rows of x, w and h (and of d_h); 0 = packed; multiples of 16 bytes */
    int64_t ld_gate_up;             /* rows of gate_up and d_gate_up: G's features, then U's; 0 = 2 features */
    int64_t ld_dx, ld_dw;
    uint32_t flags;                 /* GEMM_FLAG_CTA_GROUP_1/2, _NO_STREAM_K, _STAGE_K1/K2 as in gemm.h */
    int32_t tile_n;                 /* gates and ups of a tile together: 128, 256 or 512; 0 = planner */
    int32_t stages, max_ctas;       /* as in gemm.h; 0 = planner.  Any of these three or of the flags keeps to the persistent
                                       pipeline, and applies to the forward pass alone */
    uint64_t wait_timeout_ns;       /* bound on every device-side wait; 0 = 2 s */
} gated_desc_t;

typedef struct {
    gemm_plan_info_t product;       /* the forward pass (N = 2 features) */
    gemm_plan_info_t dx, dw;        /* the backward pass's products; zeros without gradients */
    int32_t few_tiles;              /* 1: up to 128 tokens, one wave of CTAs (gated_few.cu); otherwise the persistent pipeline */
    int32_t k_split;                /* few tiles: CTAs (one cluster) that share K */
    int64_t workspace_bytes;        /* device memory of the plan's products */
} gated_plan_info_t;

typedef struct gated_plan_s* gated_plan_t;

/* gated_plan_create -- plan on the current device.  GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_RESOURCES,
 * GEMM_ERR_NO_DEVICE or GEMM_ERR_CUDA. */
gemm_status_t gated_plan_create(gated_plan_t* plan, const gated_desc_t* desc);
gemm_status_t gated_plan_info(gated_plan_t plan, gated_plan_info_t* info);

/* gated_run -- enqueue the forward pass.  gate_up: G and U for the backward pass, [tokens][ld_gate_up], or NULL.  Pointers are
 * 16-byte aligned.  A device-side wait that ran out is reported by gated_sync_status. */
gemm_status_t gated_run(gated_plan_t plan, const void* x, const void* w, void* h, void* gate_up, gemm_stream_t stream);

/* gated_backward -- from d_h and the forward pass's x, w and gate_up: d_gate_up = [d_h U act'(G), d_h act(G)] (rounded to dtype: the
 * tensor core multiplies 16-bit operands), d_x = d_gate_up W, d_w = d_gate_up^T X.  d_gate_up may be gate_up itself; d_x or d_w
 * NULL: not wanted. */
typedef struct {
    const void* d_h;
    const void* x;
    const void* w;
    const void* gate_up;
    void* d_gate_up;
    void* d_x;                      /* [tokens][k] */
    void* d_w;                      /* [2 features][k]; tokens 0: zeroed */
} gated_grads_t;
gemm_status_t gated_backward(gated_plan_t plan, const gated_grads_t* args, gemm_stream_t stream);
gemm_status_t gated_sync_status(gated_plan_t plan, gemm_stream_t stream, gemm_device_error_t* out);
gemm_status_t gated_plan_destroy(gated_plan_t plan);

/* ------------------------------------------------------------------ products of a few tokens with 4-bit weights */

/* p[m, j] = sum over groups g of scales[j, g] * sum over k in g of x[m, k] (code[j, k] - zero[j, g]);  group g is K's elements
 * [g * group, (g + 1) * group), the last one cut short by k.  activation GATED_NONE: y = p (n columns of n weight rows).
 * Otherwise w has 2 n rows, gates first: y[m, j] = act(p[m, j]) * p[m, n + j].  Codes are 0..15, two a byte, element k in the
 * low half of byte k/2 when k is even.  Products of codes are exact; their sums, the zero points'
 * part, which is taken off a group's sum, and the scaling are fp32; y is rounded once.
 * Infinities and NaN of x and of the scales stay with their token or weight row (an infinite x gives NaN or infinities).  A bf16 x
 * past 2^63 counts as infinite, and one under 2^-57 may lose bits; so does a result for bf16 x under about 2^-70, as its sum is
 * held in steps of 2^-69. */
typedef struct {
    int32_t tokens;             /* 0 (no-op) .. 16; more go through the product, with the weights in another form */
    int32_t n, k;               /* n 1..2^30; k even, and such that X fits the shared memory of a cluster: 94208 and less does for up
                                   to 8 tokens, 45056 and less for more */
    int32_t group;              /* a multiple of 32 */
    int32_t dtype;              /* GEMM_BF16 or GEMM_F16: x, scales and y */
    int32_t activation;         /* gated_activation_t */
    const void* x;              /* rows 16-byte aligned */
    const void* codes;          /* [n or 2 n] rows of k/2 bytes, 16-byte aligned */
    const void* scales;         /* [n or 2 n][ceil(k / group)] */
    const uint8_t* zeros;       /* [n or 2 n][ceil(k / group)], 0..127, or NULL: 8 */
    void* y;                    /* [tokens][n] */
    int64_t ldx, ld_codes /* bytes */, ld_scales, ld_zeros, ldy;     /* 0 = packed */
} int4_matmul_args_t;

/* int4_matmul_run -- enqueue.  GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED (17 tokens or more, an odd or too long k, a group
 * that is no multiple of 32), GEMM_ERR_ALIGNMENT, GEMM_ERR_NO_DEVICE or GEMM_ERR_CUDA. */
gemm_status_t int4_matmul_run(const int4_matmul_args_t* args, gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_BLACKWELL_GB300_FEEDFORWARD_H */
