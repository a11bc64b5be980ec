/*
 * echo_fp8.h -- C ABI of libecho, third part: the layer operators of
 * echo_layer.h in 8-bit floating point.
 *
 * A matrix in 8 bits is a matrix of codes with one binary32 scale for each block
 * of 128, as the all-reduce's messages have one for each group of 128: an
 * element's value is its code times its block's scale.  A block is 1 x 128, along
 * a row (activations, their checkpoints, gradients), or 128 x 128 (weights).  The
 * codes are e4m3 (4 exponent bits, 3 of the fraction, largest 448, no infinity) or
 * e5m2 (5 and 2, largest 57344).
 *
 * Conventions are those of echo.h and echo_layer.h, and:
 *   - Codes stand in rows: base addresses are 16-byte aligned and row pitches
 *     multiples of 16 (ECHO_ERR_ALIGNMENT), 0 for the row's length rounded up to
 *     16.  What lies between a row's end and its pitch is not written and has no
 *     influence, whatever it holds.
 *   - Scales are dense and 4-byte aligned.  Blocks are counted from the matrix's
 *     first row and column; a last block may be short.  Of 1 x 128 blocks a row
 *     has ceil(cols / 128) scales; of 128 x 128 blocks the scales are a matrix of
 *     ceil(rows / 128) rows of ceil(cols / 128).  In a matrix of two parts (a gated
 *     product's weights, one part above the other, or its sums p, one beside the
 *     other) the second part's blocks begin anew at its first row or column.
 *   - Any binary32 scale is taken.  The matrix cores apply scales that are powers
 *     of two by themselves, so echo_linear8 is faster where all of a tile's are;
 *     otherwise a block's sum is multiplied by the two scales' product and added to
 *     the others' in binary32.  Both are the sums described below, but their last
 *     bits may differ: those of a row depend on the kind of its neighbours' scales.
 *     Of a scale of x and one of w the product must not overflow.  Below 2^-126 it
 *     may lose digits, down to 0, as binary32 numbers there do: off by at most 2^-150,
 *     times a block's sum of products of codes less than 2^-125 with x in e4m3,
 *     2^-118 in e5m2.
 *   - echo_linear8's sums are binary32 with one exception, the matrix cores' own:
 *     they add the products of eight neighbours of the contraction (8 q to 8 q + 7)
 *     after cutting each towards zero at 2^(E - 13), E the largest sum of the two
 *     codes' exponents among the eight, a subnormal code's counted as the smallest
 *     normal one's (-6 in e4m3, -14 in e5m2).  So each is off by less than 2^(E - 13),
 *     which is 2^-13 of the largest beside it where that one's codes are normal, and
 *     can be more than that where they are not.  For normal values the sum is off by
 *     2^-16 of its norm, where a rounding to half or bfloat16 is 2^-12 or 2^-9. */
#ifndef ECHO_FP8_H
#define ECHO_FP8_H

#include "echo_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ECHO_E4M3 3
#define ECHO_E5M2 4
#define ECHO_FP8_BLOCK 128 /* elements along a block's side */

/* A matrix and its 8-bit form. */
typedef struct echo_pack8_desc {
  int64_t rows, cols; /* each may be 0; rows <= ECHO_MAX_ROWS, cols <= ECHO_MAX_PITCH, their product
                         <= ECHO_MAX_PRODUCT; with blocks rows <= ECHO_MAX_PITCH too */
  int64_t ld_x;       /* row pitch of the matrix itself */
  int64_t ld_c;       /* row pitch of its codes */
  int64_t ld_t;       /* row pitch of the transposed codes */
  int32_t dtype;      /* of the matrix: ECHO_BF16, ECHO_F16 or ECHO_F32 */
  int32_t format;     /* of the codes: ECHO_E4M3 or ECHO_E5M2 */
  int32_t blocks;     /* 0: blocks of 1 x 128, 1: of 128 x 128 */
  int32_t parts;      /* 1 or 2 equal parts: of the columns, or with blocks of the rows */
} echo_pack8_desc;

/* codes = x / s rounded to nearest even and scales = s, for each block the least
 * power of two s that brings its largest finite magnitude within the codes' range
 * (1 for a block of zeros, 2^-126 at least).  A power of two costs a floating-point
 * code no digit, and code times scale is then exact in 16 bits.  NaN gives NaN;
 * inf gives NaN in e4m3 and inf in e5m2; neither has a part in its block's scale.
 * codes_t and scales_t (both NULL or both given; blocks 1, and parts 1 or parts of
 * a multiple of 128 rows, else ECHO_ERR_SHAPE) are the transposed matrix's: codes
 * cols rows of `rows`, scales ceil(cols / 128) rows of ceil(rows / 128). */
int echo_pack8(const echo_pack8_desc* d, const void* x, void* codes, float* scales, void* codes_t,
               float* scales_t, echo_stream_t stream);

/* x = codes times scales, rounded once to dtype.  A finite code's value past dtype's
 * range becomes dtype's largest number, so that one next to it, rounded up when it
 * was packed, comes back finite.  ld_t is not looked at. */
int echo_unpack8(const echo_pack8_desc* d, const void* codes, const float* scales, void* x,
                 echo_stream_t stream);

/* echo_linear's product and gradients (p = x w^T + bias, out = act(p) + residual,
 * gated out = act(p_gate) (.) p_up + residual) with operands in 8 bits. */
typedef struct echo_linear8_desc {
  int64_t m, n, k;  /* as in echo_linear_desc */
  int64_t ld_x;     /* row pitch of x's codes */
  int64_t ld_w;     /* row pitch of w: its codes, in echo_linear_backward8 its elements */
  int64_t ld_out;   /* row pitch of out, and of its gradient */
  int64_t ld_r;     /* row pitch of residual */
  int64_t ld_p;     /* row pitch of p's codes, in echo_linear_backward8 */
  int32_t dtype;    /* of every tensor that is not codes: ECHO_BF16 or ECHO_F16 */
  int32_t act;      /* ECHO_ACT_* */
  int32_t gated;    /* 0 or 1 */
  int32_t x_format; /* ECHO_E4M3 or ECHO_E5M2; w and p are e4m3 */
} echo_linear8_desc;

/* Bytes of workspace echo_linear8 needs for this shape (0 for many), or a
 * negative ECHO_ERR_*. */
int64_t echo_linear8_workspace(const echo_linear8_desc* d);

/* The forward product of x in blocks of 1 x 128 and w in blocks of 128 x 128
 * (gated, of two parts).  sx, sw: their scales.  bias (the rows of w), residual and
 * p (dense [m, rows of w], the sums with bias before the activation) may be NULL
 * and are of dtype, as out is.  out may equal residual exactly.  Gradients with
 * respect to x in 8 bits are this call again, on the packed gradient of p and the
 * transposed weights of echo_pack8. */
int echo_linear8(const echo_linear8_desc* d, const void* x, const float* sx, const void* w,
                 const float* sw, const void* bias, const void* residual, void* out, void* p,
                 void* workspace, int64_t workspace_bytes, echo_stream_t stream);

/* Bytes of workspace echo_linear_backward8 needs, whichever of its outputs are
 * asked for, or a negative ECHO_ERR_*. */
int64_t echo_linear_backward8_workspace(const echo_linear8_desc* d);

/* echo_linear_backward from checkpoints in 8 bits: x and p, the forward call's
 * input and its sums before the activation, as codes and scales in blocks of 1 x
 * 128 (gated, p of two parts); dout, w and the gradients are of dtype.
 *   dp = dout (.) act'(p), or, gated, (dout (.) p_up (.) act'(p_gate),
 *        dout (.) act(p_gate));  dx = dp w;  dw = dp^T x;  dbias = sum of dp
 * p and sp are read unless act is NONE and gated 0 (then they may be NULL).  The
 * product for dw reads x unpacked to dtype, as echo_unpack8 has it: exact for
 * scales of echo_pack8 (but for bits below half's smallest number), one more
 * rounding for others.  Everything else is as in echo_linear_backward. */
int echo_linear_backward8(const echo_linear8_desc* d, const void* dout, const void* x,
                          const float* sx, const void* w, const void* p, const float* sp, void* dx,
                          void* dw, void* dbias, void* workspace, int64_t workspace_bytes,
                          echo_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif
