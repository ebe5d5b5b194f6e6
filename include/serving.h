/*
 * serving.h -- C ABI of the operators that stand between the products of an
 * attention block, next to gemm.h and in the same library:
 *
 *   lora_*          a shared projection with the low-rank adapter of each
 *                   token's request:  Y[m] = X[m] W^T + s_i (X[m] A_i^T) B_i^T
 *   qk_norm_rope_*  RMS norm of every query and key head and its rotary
 *                   position in one pass, optionally into the slots of a paged
 *                   key-value cache; and the backward pass
 *   paged_attn_*    attention of one new token per sequence over that cache,
 *                   split over the cache's length and joined
 *
 * Conventions are gemm.h's: every call returns a gemm_status_t and nothing
 * throws across the ABI; the caller owns every buffer and the stream; calls
 * only enqueue work (no allocation, no synchronisation), so they may be
 * captured into a CUDA graph; unsupported requests fail with
 * GEMM_ERR_UNSUPPORTED, never a silent fallback.  Strides and leading
 * dimensions count elements.  Work goes to the current device; a plan runs on
 * the device it was made on (GEMM_ERR_INVALID_ARG where another one is current),
 * and all buffers lie there.  A plan may be run on one stream, from one host
 * thread, at a time (its launches share its workspace); launches of one plan
 * on several streams must be ordered by events.
 *
 * Device data is not validated on the host.  Indices read on the device
 * (adapter numbers, positions, slots, block tables, lengths) are bounds-checked
 * there: an index out of range never reads or writes outside the buffers
 * described here; what it does instead is said at each operator.
 */
#ifndef DENSE_GEMM_BLACKWELL_GB300_SERVING_H
#define DENSE_GEMM_BLACKWELL_GB300_SERVING_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ low-rank adapters beside a projection */

/* Y[m, n] = sum_k X[m, k] W[n, k] + scale[i] sum_r T[m, r] B_i[n, r],
 * T[m, r] = sum_k X[m, k] A_i[r, k], i = adapter[m]; a token with i < 0 (or i >= adapters) takes the projection alone.
 * All sums are fp32, Y is rounded once.  scale[i] T is rounded to the input type before its product with B_i (the tensor
 * core multiplies 16-bit operands); for fp32 outputs it is carried as the sum of two such values.  For f16 inputs a scale[i] T
 * past 65504 so becomes an infinity, and the token's outputs with it.  Infinities and NaN of
 * a token or of A_i and B_i stay with that token and the tokens of adapter i; many of them in B_i are slow, as the
 * outputs of other tokens beside them are computed twice. */
typedef struct {
    int64_t tokens, n, k;       /* X is tokens x k, W is n x k, Y is tokens x n; n, k >= 1; tokens 0 = no-op */
    int32_t rank;               /* rows of every A_i: a multiple of 8 in 8..256 (pad smaller ranks with zeros) */
    int32_t adapters;           /* number of adapters, 1..4096 */
    int32_t dtype;              /* X, W, A, B: GEMM_BF16 or GEMM_F16 */
    int32_t dtype_y;            /* GEMM_F32, GEMM_BF16 or GEMM_F16 */
    int64_t ldx, ldw, ldy;      /* 0 = packed (k, k, n); multiples of 16 bytes */
    uint32_t flags;             /* GEMM_FLAG_CTA_GROUP_1/2, _NO_STREAM_K, _STAGE_K1/K2 as in gemm.h */
    int32_t tile_n, stages, max_ctas;   /* as in gemm.h; 0 = planner.  Any of these or of the flags
                                   keeps to the persistent kernel where few tiles would take the few-tile one */
    uint64_t wait_timeout_ns;   /* bound on every device-side wait; 0 = 2 s */
} lora_desc_t;

typedef struct {
    gemm_plan_info_t product;   /* how the projection runs (the few-tile kernel: tiles of 128 rows, one accumulator) */
    int32_t steps_per_adapter;  /* K = 16 matrix instructions an adapter adds to a tile */
    int32_t max_adapters_per_tile;
    int32_t shrink_k_split;     /* CTAs (one cluster) that share the K range of X A_i^T */
    int32_t shrink_grid;        /* CTAs of the kernel that computes T */
    int32_t product_k_split;    /* few-tile kernel: CTAs (one cluster) that share a tile's K; otherwise 1 */
    int32_t reserved0;
    int64_t workspace_bytes;    /* device memory of the plan, the product's included */
} lora_plan_info_t;

typedef struct lora_plan_s* lora_plan_t;

/* lora_plan_create -- plan on the current device; allocates the workspace that holds T by tile and adapter
 * (tiles x min(adapters, tile rows) x tile rows x rank elements, twice that for fp32 outputs).
 * Returns GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_RESOURCES, GEMM_ERR_NO_DEVICE or GEMM_ERR_CUDA. */
gemm_status_t lora_plan_create(lora_plan_t* plan, const lora_desc_t* desc);
gemm_status_t lora_plan_info(lora_plan_t plan, lora_plan_info_t* info);

/* One run's buffers: device pointers, 16-byte aligned; the adapters' strides multiples of 16 bytes (0 = packed). */
typedef struct {
    const void* x;
    const void* w;
    const void* a;              /* A_i[r, k] at a[i * stride_a + r * lda + k] */
    int64_t lda, stride_a;
    const void* b;              /* B_i[n, r] at b[i * stride_b + n * ldb + r] */
    int64_t ldb, stride_b;
    const int32_t* adapter;     /* [tokens] */
    const float* scale;         /* [adapters] or NULL (ones) */
    void* y;                    /* must not overlap the inputs */
} lora_args_t;

/* lora_run -- enqueue the product.  Returns GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_ALIGNMENT or GEMM_ERR_CUDA; a
 * device-side wait that ran out is reported by lora_sync_status. */
gemm_status_t lora_run(lora_plan_t plan, const lora_args_t* args, gemm_stream_t stream);
gemm_status_t lora_sync_status(lora_plan_t plan, gemm_stream_t stream, gemm_device_error_t* out);
gemm_status_t lora_plan_destroy(lora_plan_t plan);

/* ------------------------------------------------------------------ head norms and rotary positions */

/* For every token t and every query and key head row x of head_dim elements:
 *   n = x * rsqrt(mean(x^2) + eps) * weight      (norm = 0: n = x; a NULL weight: ones)
 *   the first rot_dim elements of n are rotated in pairs (a, b):  a' = a c - b s,  b' = a s + b c
 *   with c = table[p][0][i], s = table[p][1][i], p = positions[t]; pair i is elements (i, i + rot_dim/2), or
 *   (2i, 2i + 1) when interleaved.  The rest of n passes through.
 * All in fp32, one rounding at the end.  positions are clamped to [0, table_rows). */
typedef struct {
    int32_t tokens, heads, kv_heads, head_dim;  /* head_dim: a multiple of 8 up to 256; heads, kv_heads >= 0 */
    int32_t rot_dim;            /* even, 0..head_dim */
    int32_t interleaved;        /* 0: halves, 1: neighbours */
    int32_t norm;               /* 0: no norm (rotation only) */
    int32_t dtype;              /* GEMM_BF16 or GEMM_F16: rows and weights */
    float eps;
    int32_t table_rows;         /* positions the table covers */
    const float* table;         /* [table_rows][2][rot_dim / 2] cos, sin */
    const int32_t* positions;   /* [tokens] */
    const void* q_weight;       /* [head_dim] or NULL */
    const void* k_weight;
    const void* q;              /* q[t * q_token + h * q_head + e]; rows 16-byte aligned */
    const void* k;
    int64_t q_token, q_head, k_token, k_head;
    void* q_out;                /* may be q itself (same strides) */
    void* k_out;                /* or NULL; may be k itself */
    int64_t q_out_token, q_out_head, k_out_token, k_out_head;
    /* cache append, when k_cache is given: token t's rotated keys, and its values v, go to slot slots[t], i.e. page
     * slots[t] / page_size, place slots[t] % page_size; a slot outside [0, num_pages * page_size) is skipped.  An
     * E4M3 cache holds round(x / scale), saturated to +-448. */
    const void* v;
    int64_t v_token, v_head;
    void* k_cache;
    void* v_cache;
    int64_t k_page, k_place, k_chead, v_page, v_place, v_chead;   /* strides of page, place in the page, head */
    const int32_t* slots;       /* [tokens] */
    int64_t num_pages;
    int32_t page_size;
    int32_t dtype_cache;        /* the rows' dtype or GEMM_E4M3 */
    float k_scale, v_scale;     /* E4M3 caches only */
} qk_norm_rope_args_t;

/* qk_norm_rope_run -- enqueue the forward pass.  GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_ALIGNMENT
 * (a pointer or stride off 16 bytes, 8 for E4M3 cache rows) or GEMM_ERR_CUDA. */
gemm_status_t qk_norm_rope_run(const qk_norm_rope_args_t* args, gemm_stream_t stream);

/* qk_norm_rope_backward -- gradients of the rows and weights.  Uses the forward's descriptive fields, table, positions,
 * weights, q and k (the forward's inputs; the forward's statistics are recomputed); q_out / k_out and the cache fields
 * are ignored.  dq_out and dk_out are the incoming gradients, dq and dk the outgoing ones (dq may be dq_out, same
 * strides); dq_weight / dk_weight: fp32 [head_dim], NULL when the weight is NULL or its gradient is not wanted.  The weight
 * gradients are summed in a fixed order.  workspace: qk_norm_rope_backward_workspace() bytes, 16-byte aligned, needed when
 * a weight gradient is asked for. */
typedef struct {
    const void* dq_out;
    const void* dk_out;
    int64_t dq_out_token, dq_out_head, dk_out_token, dk_out_head;
    void* dq;
    void* dk;
    int64_t dq_token, dq_head, dk_token, dk_head;
    float* dq_weight;
    float* dk_weight;
    void* workspace;
    int64_t workspace_bytes;
} qk_norm_rope_grads_t;
gemm_status_t qk_norm_rope_backward(const qk_norm_rope_args_t* args, const qk_norm_rope_grads_t* grads,
                                    gemm_stream_t stream);
int64_t qk_norm_rope_backward_workspace(void);

/* ------------------------------------------------------------------ attention of one token over a paged cache */

typedef struct {
    int32_t max_batch;          /* sequences of one run, at most */
    int32_t heads, kv_heads;    /* heads a multiple of kv_heads; query head h reads kv head h / (heads / kv_heads) */
    int32_t head_dim;           /* a multiple of 8 (16 for an E4M3 cache) up to 256 */
    int32_t page_size;          /* tokens per page, any >= 1 */
    int32_t dtype;              /* q and out: GEMM_BF16 or GEMM_F16 */
    int32_t dtype_cache;        /* dtype, or GEMM_E4M3 */
    int32_t window;             /* > 0: only the last `window` positions; 0: all */
    int32_t max_ctas;           /* cap on the grid; 0 = what the device holds at once */
} paged_attn_desc_t;

typedef struct {
    int32_t grid;               /* CTAs launched */
    int32_t tile_tokens;        /* cache positions of one unit of work */
    int32_t head_groups;        /* query-head groups a kv head is read for */
    int32_t smem_bytes;
    int64_t workspace_bytes;    /* device memory of the plan: partial results and counters */
} paged_attn_plan_info_t;

typedef struct paged_attn_plan_s* paged_attn_plan_t;

gemm_status_t paged_attn_plan_create(paged_attn_plan_t* plan, const paged_attn_desc_t* desc);
gemm_status_t paged_attn_plan_info(paged_attn_plan_t plan, paged_attn_plan_info_t* info);

/* out[b, h] = sum_j softmax_j(scale q[b, h] . K_j) V_j over positions j in [max(0, n - window), n), n = lengths[b] (clamped
 * to [0, table_width * page_size]); position j lies in page block_table[b][j / page_size].  K_j and V_j are the cache's
 * values times k_scale and v_scale.  lse[b, h] (NULL: not wanted) = log sum_j exp(scale q . K_j).  n = 0 gives zeros and
 * lse -inf.  Cache contents past n, or before the window, are not read into the result whatever they hold.  A page
 * number outside [0, num_pages) makes its positions count as masked; columns may name one page more than once.
 * Scores, the softmax's statistics and all sums are fp32; out is rounded once.  The tensor core multiplies 16-bit
 * operands, so the probabilities are rounded before their product with V: to bf16, or to f16 (2^15 times the
 * probability) for f16 queries and for E4M3 caches, whose values are exact in f16.  bf16 queries over an E4M3 cache
 * are scaled per head by a power of two to f16: elements under 2^-14 of the head's largest lose bits, at most 2^-24 of
 * that largest each. */
typedef struct {
    int32_t batch;
    int32_t table_width;        /* columns of the block table */
    const void* q;              /* q[b * q_batch + h * q_head + e] */
    int64_t q_batch, q_head;
    const void* k_cache;
    const void* v_cache;
    int64_t k_page, k_place, k_head, v_page, v_place, v_head;
    int64_t num_pages;
    const int32_t* block_table; /* [batch][table_width], rows table_stride apart */
    int64_t table_stride;
    const int32_t* lengths;     /* [batch] */
    void* out;
    int64_t out_batch, out_head;
    float* lse;                 /* [batch][heads] or NULL */
    float scale, k_scale, v_scale;
} paged_attn_args_t;

gemm_status_t paged_attn_run(paged_attn_plan_t plan, const paged_attn_args_t* args, gemm_stream_t stream);
gemm_status_t paged_attn_plan_destroy(paged_attn_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_BLACKWELL_GB300_SERVING_H */
