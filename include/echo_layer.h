/*
 * echo_layer.h -- C ABI of libecho, second part: the layer operators that a
 * rank runs on both sides of the all-reduce of echo.h.
 *
 * A tensor-parallel layer's all-reduce stands "between two dependent matrix
 * multiplications" ("Tensor-parallel traffic drops to 4 bits",
 * Interpretation).  These calls are what a rank runs around it on its own
 * tensors: the product before it (echo_linear), the norms after and before a
 * block with the block's gate and residual scale (echo_norm), the product
 * behind it, and their gradients for training.
 *
 * Conventions beyond those of echo.h:
 *   - Matrices are row-major with unit stride along a row; the row pitches
 *     that a descriptor names are in elements, at least the row's length, 0
 *     for exactly the row's length.  Every other tensor is dense.
 *   - Base addresses need the alignment of one element only (stats and
 *     workspace: 4 and 16 bytes).  16-byte aligned bases and row pitches that
 *     are multiples of 16 bytes are faster.
 *   - Sums, statistics and everything between reading an input and writing an
 *     output are binary32; each output is rounded once, to nearest even.
 *     One exception: the products of echo_linear_backward read the gradient of
 *     the pre-activation, dp, rounded to `dtype`, the matrix cores' operand type:
 *     one more rounding in every term of dx and dw (not of dbias).  In half
 *     precision its range counts too: a dp past 65504 is infinite, one below
 *     2^-14 keeps fewer digits.  dx, dw and dbias are linear in dout, so a
 *     caller's power-of-two scale on dout moves dp within the range, as it does
 *     for dx and dw themselves.
 *   - No atomics: the same inputs give the same bits on every call.
 *   - inf and NaN go through as the formulas have them: a row that holds one
 *     spoils that row of the norms and nothing else, an operand of a product
 *     spoils the sums that it enters.
 *   - Aliasing is judged by the byte range from a tensor's first element to
 *     its last, whatever the pitch. */
#ifndef ECHO_LAYER_H
#define ECHO_LAYER_H

#include "echo.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ECHO_BF16 0
#define ECHO_F16 1
#define ECHO_F32 2 /* norms only */

#define ECHO_NORM_NONE 0  /* N(v) = v */
#define ECHO_NORM_RMS 1   /* N(v) = v / sqrt(mean(v^2) + eps) * w + b */
#define ECHO_NORM_LAYER 2 /* N(v) = (v - mean(v)) / sqrt(var(v) + eps) * w + b */

#define ECHO_ACT_NONE 0
#define ECHO_ACT_RELU 1      /* max(p, 0) */
#define ECHO_ACT_GELU 2      /* p (1 + erf(p / sqrt 2)) / 2 */
#define ECHO_ACT_GELU_TANH 3 /* p (1 + tanh(sqrt(2/pi) (p + 0.044715 p^3))) / 2 */
#define ECHO_ACT_SILU 4      /* p / (1 + exp(-p)) */

#define ECHO_MAX_HIDDEN 16384             /* row length of the norms */
#define ECHO_MAX_PITCH (INT64_C(1) << 21) /* any row pitch; k and the rows of w of the products */
#define ECHO_MAX_ROWS (INT64_C(1) << 31)  /* tokens; m of the products */
#define ECHO_MAX_PRODUCT (INT64_C(1) << 42) /* m times k, m times the rows of w */

/* The norms around a block: u = N_post(y) on the block's output y, the
 * residual update h' = h + scale * gate (.) u, and z = N_pre(h') for the next
 * block, per token (row). */
typedef struct echo_norm_desc {
  int64_t tokens, hidden; /* tokens may be 0; 1 <= hidden <= ECHO_MAX_HIDDEN */
  int64_t ld_y;           /* row pitch of y */
  int64_t ld_h;           /* row pitch of h and of h_out */
  int64_t gate_rows;      /* 0: no gate (gate = 1).  Otherwise the gate has gate_rows rows of
                             hidden elements, tokens % gate_rows == 0, and token t uses row
                             t / (tokens / gate_rows): 1 row is a gate per channel, one row
                             per sequence or per token are the other uses */
  int32_t dtype;          /* of y, z, gate, weights, biases and their gradients */
  int32_t stream_dtype;   /* of h, h_out, dh_out, dh: dtype or ECHO_F32 */
  int32_t post, pre;      /* ECHO_NORM_* of N_post and N_pre */
  float scale;            /* residual scale */
  float eps;              /* of both norms, >= 0 */
} echo_norm_desc;

/* h_out = h + scale * gate (.) N_post(y); z = N_pre(h_out), N_pre taken of the
 * binary32 value before h_out's rounding.  w_* NULL is a weight of ones, b_*
 * NULL a bias of zeros (weights and biases of a norm that is NONE must be
 * NULL).  y NULL (then post is NONE, gate_rows 0 and h_out NULL) leaves z =
 * N_pre(h), a model's first norm; z is NULL exactly if pre is NONE; h_out NULL
 * skips that output.  stats (nullable) float[4 * tokens]: the post norm's means,
 * its reciprocal deviations, the pre norm's means and reciprocal deviations,
 * one plane of `tokens` each (mean 0 for RMS; 0 and 1 for NONE), as the
 * backward call needs them.  h_out may equal h exactly (in place). */
int echo_norm(const echo_norm_desc* d, const void* h, const void* y, const void* gate,
              const void* w_post, const void* b_post, const void* w_pre, const void* b_pre,
              void* h_out, void* z, float* stats, echo_stream_t stream);

/* Bytes of workspace echo_norm_backward needs (0 for tokens < 1); negative
 * ECHO_ERR_SHAPE if the descriptor's shape is refused. */
int64_t echo_norm_backward_workspace(const echo_norm_desc* d);

/* Gradients of echo_norm from dz (gradient of z, dense) and dh_out (gradient
 * of h_out from the rest of the stream, dense, NULL for none), with the
 * forward call's inputs, its h_out and its stats:
 *   dh     = dh_out + N_pre'(dz)             (dense, stream_dtype)
 *   dy     = N_post'(scale * gate (.) dh)    (dense, dtype; NULL to skip)
 *   dgate  = sum over the gate row's tokens of scale * u (.) dh
 *   dw, db = sums over the tokens, per channel
 * Parameter gradients (dtype) may be NULL to skip them; asked for, they are
 * written whole, zeros where there are no tokens.  h_out is read where pre is
 * not NONE, y where post is not NONE or dgate is wanted; dz is NULL exactly if
 * pre is NONE.  dh may equal dh_out exactly. */
int echo_norm_backward(const echo_norm_desc* d, const void* dz, const void* dh_out,
                       const void* h_out, const void* y, const float* stats, const void* gate,
                       const void* w_post, const void* b_post, const void* w_pre, void* dh,
                       void* dy, void* dgate, void* dw_post, void* db_post, void* dw_pre,
                       void* db_pre, void* workspace, int64_t workspace_bytes,
                       echo_stream_t stream);

/* A matrix product with its epilogue: p = x w^T + bias and out = act(p) +
 * residual, or, gated, out = act(p_gate) (.) p_up + residual.  x is m rows of
 * k, out m rows of n, w n rows of k: row j holds the weights of output j.
 * Gated, w has 2n rows, the gate's first and the up rows behind them; bias,
 * p, and the gradients of w and bias have the same order. */
typedef struct echo_linear_desc {
  int64_t m, n, k;   /* each may be 0; m <= ECHO_MAX_ROWS, k and the rows of w <= ECHO_MAX_PITCH,
                        m k and m times the rows of w <= ECHO_MAX_PRODUCT (8 TiB, more than
                        a device holds) */
  int64_t ld_x;      /* row pitch of x */
  int64_t ld_w;      /* row pitch of w */
  int64_t ld_out;    /* row pitch of out, and of its gradient */
  int64_t ld_r;      /* row pitch of residual */
  int32_t dtype;     /* of every tensor: ECHO_BF16 or ECHO_F16 */
  int32_t act;       /* ECHO_ACT_* */
  int32_t gated;     /* 0 or 1 */
  int32_t reserved;  /* 0 */
} echo_linear_desc;

/* Bytes of workspace echo_linear needs for this shape (0 for many), or a
 * negative ECHO_ERR_*. */
int64_t echo_linear_workspace(const echo_linear_desc* d);

/* The forward product.  bias (the rows of w), residual [m, n] and p (dense
 * [m, rows of w]: the sums with bias before the activation, kept for the
 * backward call) may be NULL.  out may equal residual exactly. */
int echo_linear(const echo_linear_desc* d, const void* x, const void* w, const void* bias,
                const void* residual, void* out, void* p, void* workspace,
                int64_t workspace_bytes, echo_stream_t stream);

/* Bytes of workspace echo_linear_backward needs, whichever of its outputs are
 * asked for, or a negative ECHO_ERR_*. */
int64_t echo_linear_backward_workspace(const echo_linear_desc* d);

/* Gradients of echo_linear from dout (pitch ld_out) and the forward call's x,
 * w and p:
 *   dp = dout (.) act'(p), or, gated, (dout (.) p_up (.) act'(p_gate),
 *        dout (.) act(p_gate));   rounded to dtype for the two products
 *   dx = dp w (dense [m, k]);  dw = dp^T x (dense, the shape of w);
 *   dbias = sum over the rows of dp (of its binary32 values)
 * The residual's gradient is dout itself.  Each of dx, dw, dbias may be NULL to
 * skip it; asked for, it is written whole, zeros where the sum is empty.  p is
 * read unless act is NONE and gated 0 (then it may be NULL). */
int echo_linear_backward(const echo_linear_desc* d, const void* dout, const void* x,
                         const void* w, const void* p, void* dx, void* dw, void* dbias,
                         void* workspace, int64_t workspace_bytes, echo_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif
