/*
 * moe_block.h -- C ABI of the feed-forward block for many tokens, forward and
 * backward (GB300, sm_103a): the gated product and the second product of
 * experts whose rows are grouped (or of one dense block), and the norms before
 * and after a block fused with its gate and residual scale.
 *
 * Conventions are those of moe_combine.h: the caller owns every buffer, the
 * library allocates nothing and keeps no state between calls, all work is
 * enqueued on `stream` and returns without synchronising, arguments are
 * validated on the host before anything is launched, and every call touches
 * global memory only after the previous kernel on the stream has completed.
 *
 * Rows and experts.  Row r belongs to expert e where offsets[e] <= r <
 * offsets[e + 1] (offsets of moe_build_row_map, rows of moe_dispatch_permute).
 * Rows before offsets[0] and from offsets[E] on belong to no expert: nothing of
 * theirs is read into a result and nothing is written.  offsets may be NULL with
 * E == 1: every row is the one expert's.  The offsets are device memory; a kernel
 * treats one that lies below its predecessor as equal to it, and one outside [0, rows]
 * as the nearer end, and records MOE_ERR_ROW_OUT_OF_RANGE in *status.
 *
 * Matrices of rows may have strides (elements from row to row); pointers are
 * 16-byte aligned and strides multiples of 8.  Outputs must not overlap inputs or
 * each other.
 *
 * Numerics.  Sums are held in fp32 and each result is rounded once to its type.
 * The order of the sums depends on the sizes and offsets alone, so a call gives
 * the same result every time.  A NaN or infinity of a row reaches that row's
 * results and its expert's weight gradient only.
 *
 * Waits inside the products' kernels are bounded.  One that runs out (after 2 s and
 * 4 us for each 64 of the contraction that is multiplied while it lasts, more than ten
 * times what a healthy launch takes) turns results that depend on it into NaN and
 * records MOE_ERR_DEVICE_TIMEOUT in *status; nothing faults or hangs.  The norms have no
 * status: a wait that runs out there (2 s) shows in NaN alone, in its row's results and in the
 * sums over tokens.
 * moe_debug_stall (moe_combine.h) stops the first thread block's copies of a product
 * and the copies of a norm's first rows after its number of steps, to test that.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (validated on the host): H, I, K and N up to MOE_BLOCK_MAX_DIM and
 * multiples of 8, E up to MOE_LAYER_MAX_EXPERTS, rows below 2^31 - 2^16, strides of the
 * products' matrices up to MOE_BLOCK_MAX_STRIDE. */
#define MOE_BLOCK_MAX_DIM 65536
#define MOE_BLOCK_MAX_STRIDE ((INT64_C(1) << 39) - 8)

/* ------------------------------------------------------------------------
 * Gated product of a feed-forward block, both projections in one kernel:
 *
 *   g[r] = W1[e] x[r],  u[r] = W3[e] x[r]        e the expert of row r
 *   out[r] = act(g[r]) * u[r]                    (elementwise, I values)
 *
 * w13 holds W1's I rows and then W3's for each expert ([E, 2 I, H], as in
 * moe_layer).  gate_up, when given, receives g and then u of each row, rounded
 * to io_dtype: what the backward pass takes.  out is computed from the unrounded
 * sums.  rows == 0 is a no-op.
 * ---------------------------------------------------------------------- */
typedef struct moe_gated_linear_args {
    int64_t rows;
    int32_t H, I, E;
    int32_t activation;       /* moe_activation */
    const int32_t *offsets;   /* device int32 [E + 1], or NULL with E == 1 */
    const void *x;            /* device [rows, H] (io_dtype) */
    int64_t x_stride;
    const void *w13;          /* device [E, 2 I, H] (io_dtype) */
    void *gate_up;            /* device [rows, 2 I] (io_dtype) or NULL */
    int64_t gate_up_stride;
    void *out;                /* device [rows, I] (io_dtype) */
    int64_t out_stride;
    int32_t *status;          /* device int32 or NULL, zeroed by the caller; the first error found */
    int32_t io_dtype;         /* moe_io_dtype */
} moe_gated_linear_args;

moe_status moe_gated_linear(const moe_gated_linear_args *args, moe_stream_t stream);
size_t moe_gated_linear_args_size(void);

/* ------------------------------------------------------------------------
 * Its gradients, from the gate_up that the forward pass left:
 *
 *   dg = d_out * u * act'(g),  du = d_out * act(g)
 *   d_x[r]   = W1[e]^T dg[r] + W3[e]^T du[r]
 *   d_w13[e] = the sum of [dg; du][r] x[r]^T over the expert's rows (0 where it has none)
 *
 * dg and du are rounded once to io_dtype between (they are the products'
 * operands): the gradients' relative error is 2.3e-3 to 2.5e-3 in bf16, of which
 * their own rounding makes 1.7e-3 (fp16: 3e-4 and 2.1e-4).  Small calls (rows <= 32 and
 * rows * (I + 56) <= 4096) hold them as sums of two io_dtype values and have that
 * rounding alone; the limits are of what it costs, not of errors, which depend little
 * on the number of rows.  In fp16, values below 2^-24 vanish there and values beyond 65504 become
 * infinities, so losses are scaled as usual.  Either of d_x and d_w13 may be NULL; w13 is
 * read for d_x only and x for d_w13 only (NULL otherwise).  With rows == 0,
 * d_w13 is set to 0 and the rest is a no-op.
 *
 * workspace: device memory of moe_gated_linear_backward_workspace_size(...)
 * bytes, 16-byte aligned, not shared by calls that may overlap; it holds dg and du
 * of every row, and what it holds before a call does not matter.  The
 * size never falls as rows grow, so one made for the largest batch serves every smaller
 * one, and is at most 32 KB more than the 4 rows I bytes of dg and du.
 * ---------------------------------------------------------------------- */
typedef struct moe_gated_linear_backward_args {
    int64_t rows;
    int32_t H, I, E;
    int32_t activation;
    const int32_t *offsets;
    const void *d_out;        /* device [rows, I] (io_dtype) */
    int64_t d_out_stride;
    const void *gate_up;      /* device [rows, 2 I] (io_dtype) */
    int64_t gate_up_stride;
    const void *x;            /* device [rows, H] (io_dtype) */
    int64_t x_stride;
    const void *w13;          /* device [E, 2 I, H] (io_dtype) */
    void *d_x;                /* device [rows, H] (io_dtype) or NULL */
    int64_t d_x_stride;
    void *d_w13;              /* device [E, 2 I, H] (grad_dtype) or NULL */
    void *workspace;
    size_t workspace_bytes;
    int32_t *status;
    int32_t io_dtype;
    int32_t grad_dtype;       /* moe_weight_dtype of d_w13: MOE_WEIGHTS_FP32, or io_dtype's own type */
} moe_gated_linear_backward_args;

moe_status moe_gated_linear_backward_workspace_size(int64_t rows, int32_t I, size_t *bytes);
moe_status moe_gated_linear_backward(const moe_gated_linear_backward_args *args, moe_stream_t stream);
size_t moe_gated_linear_backward_args_size(void);

/* ------------------------------------------------------------------------
 * Linear product of grouped rows (the block's second product):
 * out[r] = W[e] x[r], w [E, N, K].  rows == 0 is a no-op.
 * ---------------------------------------------------------------------- */
typedef struct moe_grouped_linear_args {
    int64_t rows;
    int32_t K, N, E;
    int32_t io_dtype;
    const int32_t *offsets;
    const void *x;            /* device [rows, K] (io_dtype) */
    int64_t x_stride;
    const void *w;            /* device [E, N, K] (io_dtype) */
    void *out;                /* device [rows, N] (io_dtype) */
    int64_t out_stride;
    int32_t *status;
} moe_grouped_linear_args;

moe_status moe_grouped_linear(const moe_grouped_linear_args *args, moe_stream_t stream);
size_t moe_grouped_linear_args_size(void);

/* ------------------------------------------------------------------------
 * Its gradients: d_x[r] = W[e]^T d_out[r], d_w[e] = the sum of d_out[r] x[r]^T
 * over the expert's rows (0 where it has none).  Either of d_x and d_w may be
 * NULL; w is read for d_x only and x for d_w only.  With rows == 0, d_w is set
 * to 0 and the rest is a no-op.
 * ---------------------------------------------------------------------- */
typedef struct moe_grouped_linear_backward_args {
    int64_t rows;
    int32_t K, N, E;
    int32_t io_dtype;
    const int32_t *offsets;
    const void *d_out;        /* device [rows, N] (io_dtype) */
    int64_t d_out_stride;
    const void *x;            /* device [rows, K] (io_dtype) */
    int64_t x_stride;
    const void *w;            /* device [E, N, K] (io_dtype) */
    void *d_x;                /* device [rows, K] (io_dtype) or NULL */
    int64_t d_x_stride;
    void *d_w;                /* device [E, N, K] (grad_dtype) or NULL */
    int32_t *status;
    int32_t grad_dtype;
} moe_grouped_linear_backward_args;

moe_status moe_grouped_linear_backward(const moe_grouped_linear_backward_args *args, moe_stream_t stream);
size_t moe_grouped_linear_backward_args_size(void);

/* ------------------------------------------------------------------------
 * The norms after a block and before the next one, with the block's gate and
 * the residual's scale, in one pass over the rows:
 *
 *   n = y / sqrt(mean(y^2) + eps),  a = n * (post_gamma + weight_bias)  (a = y without post_gamma)
 *   s = residual_scale * residual + block_scale * gate * a              (no gate: 1; no residual: 0)
 *   residual_out = s,  norm_out = s / sqrt(mean(s^2) + eps) * (pre_gamma + weight_bias)
 *
 * The second norm reads the unrounded s, as the combine's does.  gate has one
 * value for each channel ([H], io_dtype) or for each token ([T], fp32).
 * y is a block's output (a combine's combined_out, a grouped linear's out).
 * T rows of H elements, one after the other; residual_out may be residual or y,
 * and norm_out may be y.  H a multiple of 8, up to MOE_MAX_HIDDEN.  T == 0 is a no-op.
 * ---------------------------------------------------------------------- */
typedef enum {
    MOE_GATE_NONE = 0,
    MOE_GATE_CHANNEL = 1, /* device [H] (io_dtype) */
    MOE_GATE_TOKEN = 2    /* device fp32 [T] */
} moe_gate_kind;

typedef struct moe_block_norm_args {
    int64_t T;
    int32_t H;
    int32_t io_dtype;
    const void *y;            /* device [T, H] (io_dtype) */
    const void *residual;     /* device [T, H] (io_dtype) or NULL */
    const void *post_gamma;   /* device [H] (io_dtype) or NULL = no norm after the block */
    const void *pre_gamma;    /* device [H] (io_dtype) or NULL; norm_out needs it */
    const void *gate;         /* as gate_kind says, NULL for MOE_GATE_NONE */
    int32_t gate_kind;        /* moe_gate_kind */
    float block_scale, residual_scale; /* finite */
    float eps;                /* >= 0, inside the square roots */
    float weight_bias;        /* added to both gammas: 0 standard, 1 the (1 + gamma) form */
    void *residual_out;       /* device [T, H] (io_dtype) or NULL */
    void *norm_out;           /* device [T, H] (io_dtype) or NULL; at least one output */
} moe_block_norm_args;

moe_status moe_block_norm(const moe_block_norm_args *args, moe_stream_t stream);
size_t moe_block_norm_args_size(void);

/* ------------------------------------------------------------------------
 * Its gradients.  With ds the gradient of s (d_residual_out plus what comes
 * back through the second norm), m = s / sqrt(mean(s^2) + eps):
 *
 *   ds          = d_residual_out + (v - m mean(v m)) / sqrt(mean(s^2) + eps),
 *                 v = d_norm_out * (pre_gamma + weight_bias)
 *   d_residual  = residual_scale * ds
 *   d_gate      = the sum of block_scale * a * ds over tokens (channel) or channels (token)
 *   da          = block_scale * gate * ds
 *   d_y         = (p - n mean(p n)) / sqrt(mean(y^2) + eps), p = da * (post_gamma + weight_bias)
 *                 (da without post_gamma)
 *   d_post_gamma = sum over tokens of da * n,  d_pre_gamma = of d_norm_out * m
 *
 * s is computed again from y and residual, in fp32.  Sums over tokens are fp32
 * and in an order that T and H alone decide.  Each of d_residual_out and
 * d_norm_out may be NULL (a gradient of 0), not both; every output may be
 * NULL.  pre_gamma is needed with d_norm_out.  d_y may be y, d_residual_out or
 * d_norm_out, and d_residual may be residual, d_residual_out or d_norm_out (but d_y
 * and d_residual are not the same).  The gradients of gamma and gate are fp32 and
 * are written, not added to; with T == 0 those over tokens are 0 and the rest is a no-op.
 *
 * workspace: device memory of moe_block_norm_backward_workspace_size(T, H)
 * bytes, 16-byte aligned, not shared by calls that may overlap; not needed
 * (NULL) where no sum over tokens is asked for.
 * ---------------------------------------------------------------------- */
typedef struct moe_block_norm_backward_args {
    int64_t T;
    int32_t H;
    int32_t io_dtype;
    const void *y;
    const void *residual;     /* as in the forward pass */
    const void *post_gamma;
    const void *pre_gamma;
    const void *gate;
    int32_t gate_kind;
    float block_scale, residual_scale;
    float eps;
    float weight_bias;
    const void *d_residual_out; /* device [T, H] (io_dtype) or NULL */
    const void *d_norm_out;   /* device [T, H] (io_dtype) or NULL */
    void *d_y;                /* device [T, H] (io_dtype) or NULL */
    void *d_residual;         /* device [T, H] (io_dtype) or NULL; needs residual */
    float *d_post_gamma;      /* device fp32 [H] or NULL; needs post_gamma */
    float *d_pre_gamma;       /* device fp32 [H] or NULL; needs d_norm_out */
    float *d_gate;            /* device fp32 [H] or [T], or NULL; needs gate */
    void *workspace;
    size_t workspace_bytes;
} moe_block_norm_backward_args;

moe_status moe_block_norm_backward_workspace_size(int64_t T, int32_t H, size_t *bytes);
moe_status moe_block_norm_backward(const moe_block_norm_backward_args *args, moe_stream_t stream);
size_t moe_block_norm_backward_args_size(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
