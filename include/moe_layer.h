/*
 * moe_layer.h -- C ABI of the few-token serving operators around the MoE
 * combine (GB300, sm_103a): expert selection from router logits, a linear
 * layer with 4-bit weights, and a whole expert layer for a few tokens.
 *
 * Conventions are those of moe_combine.h: the caller owns every buffer,
 * the library allocates nothing and keeps no state between calls, all work is
 * enqueued on `stream` and returns without synchronising, arguments are
 * validated on the host before anything is launched, and every call is
 * launched with programmatic dependent launch and touches global memory only
 * after the previous kernel on the stream has completed.  Unlike the combine,
 * these operators define what non-finite values do; see each.
 *
 * Outputs must not overlap inputs, except that the layer's out may be its x,
 * shared_out or residual (with rows one after the other).
 *
 * Waits inside the kernels are bounded.  One that runs out (after 2 s, which no
 * healthy launch comes near) turns every result that depends on it into NaN;
 * the expert layer also records MOE_ERR_DEVICE_TIMEOUT in its status word.
 * Nothing faults or hangs, and the context stays usable.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_combine.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits of the few-token products (validated on the host). */
#define MOE_FEW_TOKENS 64          /* rows of x of a linear, tokens of a layer */
#define MOE_LAYER_MAX_EXPERTS 1024
#define MOE_FEW_MAX_DIM 65536      /* N of a linear, I of a layer */
#define MOE_FEW_MAX_K 32768        /* K of a linear, H of a layer */

/* How a weight matrix [rows, K] is held.  4-bit codes are packed two to a
 * byte, element 2i of a row in the low nibble of byte i, rows contiguous. */
typedef enum {
    MOE_W_16 = 0,    /* io_dtype elements; K % 8 == 0 */
    MOE_W_NVFP4 = 1, /* e2m1 codes, one e4m3 scale byte per 16 elements ([rows, K / 16],
                        linear), and a global scale g: weight = code * scale / g, the
                        convention of MOE_QUANT_NVFP4.  K % 16 == 0 */
    MOE_W_INT4 = 2   /* unsigned codes, one io_dtype scale per group_size elements
                        ([rows, K / group_size]) and optionally one uint8 zero point
                        (0..15; 8 where none are given): weight = (code - zero) * scale.
                        group_size a power of two >= 64, K % group_size == 0 */
} moe_weight_format;

typedef enum {
    MOE_SCORE_SOFTMAX = 0, /* exp(l_e) / sum over all experts */
    MOE_SCORE_SIGMOID = 1  /* 1 / (1 + exp(-l_e)) */
} moe_scoring;

typedef enum {
    MOE_ACT_SILU = 0,     /* g / (1 + exp(-g)) */
    MOE_ACT_GELU_TANH = 1 /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
} moe_activation;

/* ------------------------------------------------------------------------
 * Expert selection: for each token the top_k experts with the largest logits,
 * in descending order, and their weights.
 *
 *   topk_ids[t, j]       the expert with the j-th largest logit; equal logits
 *                        (-0 equals 0) are ordered by the lower index first
 *   router_weights[t, j] score(l) * scale, with renormalize score(l) / (sum of
 *                        the selected scores) * scale
 *
 * A logit of -inf or NaN closes the expert: it is never selected and adds
 * nothing to the softmax.  Where fewer than top_k experts are open, the slots
 * left over get id -1 and weight 0 (the padding convention of
 * moe_build_row_map and moe_layer).  A logit of +inf is selected first; the
 * softmax takes it as the largest finite float, so several share the weight.
 * Scores are computed in fp32.
 *
 * logits        device [T, E], row t at logits + t * logits_stride elements
 *               (logits_stride >= E), element type logits_dtype
 *               (moe_weight_dtype)
 * topk_ids      device int32 [T, top_k]
 * router_weights device [T, top_k], element type weight_dtype
 * Limits: 1 <= top_k <= min(MOE_MAX_TOP_K, E), E <= MOE_MAX_EXPERTS.
 * T == 0 is a no-op.
 * ---------------------------------------------------------------------- */
moe_status moe_select_experts(const void *logits, int64_t T, int32_t E, int64_t logits_stride, int32_t logits_dtype,
                              int32_t top_k, int32_t scoring, int32_t renormalize, float scale, int32_t *topk_ids,
                              void *router_weights, int32_t weight_dtype, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Linear layer with 4-bit weights for a few rows: out[m, n] = sum_k x[m, k]
 * W[n, k], rounded once from fp32.
 *
 * M rows of x, 0 <= M <= MOE_FEW_TOKENS (M == 0 is a no-op); N >= 1 rows of W.
 * x and out may have strides between their rows.  Every weight is exact: an
 * e2m1 code times its e4m3 scale is a bf16 and an fp16 number, and sums of x
 * times an int4 code less its zero point are multiplied by the scale in fp32.
 * x is exact too, but for bf16 rows with NVFP4 weights, few rows and much K:
 * these are multiplied as fp16 times a power of two for each 256 elements of a
 * row, and an element below 2^-29 of the largest of its 256 is off by up to 2^-39 of
 * that one, or by up to 2^-150 max(g, 1) if that is more.  Sums are held in fp32 in
 * an order that depends on the sizes alone (of bf16 rows with NVFP4 weights
 * otherwise at 2^-26 of the products of x, code and scale, so that they do not
 * overflow before they are divided by g: what falls below fp32's range is at most
 * 2^-123 / g a product); a result beyond io_dtype's range rounds to an infinity,
 * and a NaN or infinity of x reaches that row of out only.
 * ---------------------------------------------------------------------- */
typedef struct moe_linear_w4_args {
    int64_t M;
    int32_t N, K;
    const void *x;          /* device [M, K] (io_dtype), 16-byte aligned */
    int64_t x_stride;       /* elements from row to row of x, >= K, multiple of 8 */
    const void *w;          /* device uint8 [N, K / 2], 16-byte aligned */
    const void *w_scales;   /* device [N, K / 16] bytes (NVFP4) or [N, K / group_size] io_dtype */
    const void *w_zeros;    /* device uint8 [N, K / group_size] or NULL (INT4 only) */
    float global_scale;     /* NVFP4 g, finite > 0 (ignored otherwise) */
    int32_t w_format;       /* MOE_W_NVFP4 or MOE_W_INT4 */
    int32_t group_size;     /* INT4: see moe_weight_format; ignored otherwise */
    int32_t io_dtype;       /* moe_io_dtype of x, out and int4 scales */
    void *out;              /* device [M, N] (io_dtype) */
    int64_t out_stride;     /* elements from row to row of out, >= N */
} moe_linear_w4_args;

moe_status moe_linear_w4(const moe_linear_w4_args *args, moe_stream_t stream);
size_t moe_linear_w4_args_size(void);

/* ------------------------------------------------------------------------
 * A whole expert layer for a few tokens, in two kernels:
 *
 *   h[t, e]  = act(W1[e] x[t]) * (W3[e] x[t])             (elementwise, I values)
 *   out[t]   = sum_j router_weights[t, j] * W2[e_tj] h[t, e_tj]
 *              + shared_out[t] + residual[t]              (both optional)
 *
 * w13 holds W1's I rows and then W3's for each expert ([E, 2 I, H]); w2 is
 * [E, H, I].  Only the weights of experts that a token takes are read, once for
 * every part of an expert's tokens.  A part has up to 8 tokens; fewer where the
 * rows of x do not fit in shared memory, and where T * top_k slots spread thinly
 * over E experts: at most twice what an expert has on average, at least 2 (T = 64,
 * E = 256, top_k = 1: 3).  Skewed ids cost most there.  A slot with id -1 adds
 * nothing whatever its weight; other ids outside [0, E) are treated the same
 * and recorded in *status as MOE_ERR_INVALID_EXPERT.  A token may name an
 * expert more than once: its weights add up.  Tokens without any expert still
 * get shared_out + residual (or 0).
 *
 * Numerics: sums, the activation and the products are fp32; the weighted
 * gated product router_weight * h is rounded to io_dtype once between the two
 * kernels (it is the second product's operand), and out once at the end.  In
 * fp16 a weighted product beyond 65504 becomes an infinity.  With NVFP4 and bf16
 * the first product takes rows of x as the linear does with few of them, and the
 * second holds its sums as the linear does otherwise.  The result does not
 * depend on the other tokens of the batch in order or number beyond the order
 * of fp32 sums, and is the same from call to call.
 *
 * workspace: device memory of moe_layer_workspace_size(...) bytes (a row of I
 * 16-bit values, rounded up to a multiple of 256, for each of T * top_k slots),
 * 16-byte aligned, not shared by calls that may overlap; what it holds before a
 * call does not matter.  Limits: T <= MOE_FEW_TOKENS,
 * E <= MOE_LAYER_MAX_EXPERTS, top_k <= MOE_MAX_TOP_K; H and I multiples of 8
 * (16-bit weights), 16 (NVFP4) or group_size (INT4).  T == 0 is a no-op.
 * ---------------------------------------------------------------------- */
typedef struct moe_layer_args {
    int64_t T;
    int32_t H, I, E, top_k;
    const void *x;              /* device [T, H] (io_dtype), 16-byte aligned */
    int64_t x_stride;           /* elements from row to row of x, >= H, multiple of 8 */
    const int32_t *topk_ids;    /* device int32 [T, top_k], -1 = no expert */
    const void *router_weights; /* device [T, top_k] (weight_dtype) */
    const void *w13;            /* device [E, 2 I, H] in w_format, 16-byte aligned */
    const void *w13_scales;     /* device scales of w13's rows (4-bit formats) */
    const void *w13_zeros;      /* device zero points or NULL (INT4) */
    const float *w13_global;    /* device fp32 [E]: g of each expert, or NULL = 1 (NVFP4) */
    const void *w2;             /* device [E, H, I] in w_format, 16-byte aligned */
    const void *w2_scales;
    const void *w2_zeros;
    const float *w2_global;
    const void *shared_out;     /* device [T, H] (io_dtype) or NULL */
    const void *residual;       /* device [T, H] (io_dtype) or NULL */
    void *out;                  /* device [T, H] (io_dtype) */
    void *workspace;
    size_t workspace_bytes;
    int32_t *status;            /* device int32 or NULL, zeroed by the caller; the first error found */
    int32_t w_format;           /* moe_weight_format */
    int32_t group_size;         /* INT4 */
    int32_t activation;         /* moe_activation */
    int32_t io_dtype;           /* moe_io_dtype of x, 16-bit weights, int4 scales, shared_out, residual, out */
    int32_t weight_dtype;       /* moe_weight_dtype of router_weights */
} moe_layer_args;

moe_status moe_layer_workspace_size(int64_t T, int32_t top_k, int32_t I, size_t *bytes);
moe_status moe_layer(const moe_layer_args *args, moe_stream_t stream);
size_t moe_layer_args_size(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
