/*
 * residual_norm.h -- C ABI of libmeswish's border between transformer blocks for
 * AMD Instinct MI355X (gfx950): how a block's output z enters the residual
 * stream x, with the norms on either side, the gate and the scales, in one pass.
 *
 * For every row of n values:
 *
 *     p = Norm(z; w_post, b_post)   or z                       (post)
 *     y = skip x + scale gate * p
 *     o = Norm(y; w_pre, b_pre)     or absent                  (pre)
 *
 *     Norm(v; w, b) = (v - mean) rstd w + b,  mean = sum v / n  (center)
 *                                             mean = 0      (not center)
 *                     rstd = 1 / sqrt(sum (v - mean)^2 / n + eps)
 *
 * Backward, from dy and do (the gradients of y and o), y, z and the statistics
 * of the rows, with vhat = (v - mean) rstd and through(c, vhat) =
 * rstd (c - [center] sum c / n - vhat sum(c vhat) / n):
 *
 *     e  = dy + through(do w_pre, yhat)           (pre; dy alone otherwise)
 *     dx = skip e,   t = scale e
 *     q  = t gate,   dz = through(q w_post, zhat) (post; q otherwise)
 *     dgate = sum t p            over the rows that share a gate row
 *     dw_pre = sum do yhat, db_pre = sum do, dw_post = sum q zhat, db_post = sum q
 *
 * In the manner of the memory-efficient activations the backward keeps the
 * stream y, which the next block reads anyway (with pre), z (with post or for
 * dgate), and two values a row and norm.
 *
 * Conventions (as in meswish.h): device pointers owned by the caller, no
 * allocation or synchronisation, asynchronous on `stream` (a hipStream_t,
 * NULL = default stream), status codes from meswish_status, nothing
 * launched on an error.
 *   - Types: x, y, dx, dy have stream_dtype; z, o, dz, do branch_dtype; the
 *     weights, biases, the gate and their gradients param_dtype; each MESWISH_F32
 *     or MESWISH_BF16, but no bfloat16 stream with binary32 branches.  Arithmetic,
 *     statistics and sums are binary32; o is computed from y before its rounding.
 *     Every output is rounded once, to nearest even.
 *   - ld*: elements between the starts of consecutive rows, at least n; rows are
 *     contiguous.  Element alignment is required.
 *   - Results are deterministic: sums have a fixed order, no atomics.
 *   - Limits: n < 2^31.
 *   - An output may not overlap an input, another output or the workspace
 *     (MESWISH_EALIAS); column ranges of one matrix do not overlap.
 *   - rows == 0 writes zeros to the gradients of the parameters; n == 0 does
 *     nothing.
 */
#ifndef RESIDUAL_NORM_H
#define RESIDUAL_NORM_H

#include <stddef.h>

#include "meswish.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What both directions share.  At least one of post and pre is set. */
typedef struct {
    size_t rows, n;
    size_t gates; /* rows of the gate; it divides `rows`, and each of its rows
                     serves rows / gates consecutive ones (no gate: 1) */
    const void *gate;        /* [gates, n], or NULL for ones */
    const void *post_weight; /* [n] each, or NULL: ones and zeros */
    const void *post_bias;
    const void *pre_weight;
    const void *pre_bias;
    float skip, scale, eps;
    int post, pre, center;
    int stream_dtype, branch_dtype, param_dtype;
} residual_norm_op;

/* Forward.  o, ldo, pre_mean and pre_rstd only with pre, post_mean and post_rstd
 * only with post; the means only with center (what does not apply is not
 * looked at).  The statistics are binary32, [rows], and may be NULL. */
int residual_norm_fwd(const residual_norm_op *op, const void *x, size_t ldx, const void *z,
                      size_t ldz, void *y, size_t ldy, void *o, size_t ldo, float *post_mean,
                      float *post_rstd, float *pre_mean, float *pre_rstd, void *stream);

/* Bytes of workspace residual_norm_bwd needs (0: sizes out of range). */
size_t residual_norm_workspace_bytes(size_t rows, size_t n, size_t gates);

/* Backward.  y, dout (= do) and the statistics of pre only with pre, those of
 * post only with post; z only with post or dgate.  dy may be NULL with pre: zeros.  The
 * gradients of the parameters and of the gate may be NULL, each by itself: what
 * is NULL is not written.  workspace: 16-byte aligned, as large as
 * residual_norm_workspace_bytes(rows, n, gates) says. */
int residual_norm_bwd(const residual_norm_op *op, const void *y, size_t ldy, const void *z,
                      size_t ldz, const void *dy, size_t lddy, const void *dout, size_t lddout,
                      const float *post_mean, const float *post_rstd, const float *pre_mean,
                      const float *pre_rstd, void *dx, size_t lddx, void *dz, size_t lddz,
                      void *dgate, void *dpost_weight, void *dpost_bias, void *dpre_weight,
                      void *dpre_bias, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RESIDUAL_NORM_H */
