/*
 * layer_norm.h -- C ABI of libmeswish's layer normalization for AMD
 * Instinct MI355X (gfx950).
 *
 * Layer normalization over the last dimension of a matrix of `rows` rows of
 * n elements (any leading shape, flattened):
 *
 *     mean = sum_i x_i / n
 *     rstd = 1 / sqrt(sum_i (x_i - mean)^2 / n + eps)
 *     xhat_i = (x_i - mean) rstd
 *     y_i = xhat_i weight_i + bias_i                             (forward)
 *
 * and, for an upstream gradient dy, with g_i = dy_i weight_i,
 *
 *     dx_i = rstd (g_i - mean_j(g_j) - xhat_i mean_j(g_j xhat_j))
 *     dweight_i = sum over the rows of dy_i xhat_i
 *     dbias_i   = sum over the rows of dy_i                     (backward)
 *
 * The backward keeps the input and two binary32 values a row (mean, rstd);
 * the normalized map is recomputed from them.
 *
 * Conventions (as in meswish.h): device pointers owned by the caller, no
 * allocation or synchronisation, asynchronous on `stream` (a hipStream_t,
 * NULL = default stream), status codes from meswish_status, nothing
 * launched on an error.
 *   - dtype: MESWISH_F32 or MESWISH_BF16 for x, y, dy, dx; param_dtype the
 *     same for weight, bias, dweight, dbias (any combination).  mean, rstd:
 *     binary32.  Arithmetic, statistics and reductions are binary32; each
 *     output is rounded once, to nearest even.
 *   - ld*: elements between the starts of consecutive rows, >= n.  Rows are
 *     contiguous.  Element alignment is required, no more; rows whose start
 *     is 16-byte aligned move a little faster.
 *   - Results are deterministic: reductions have a fixed order.
 *   - Limits: n < 2^31; (rows - 1) ld + n < 2^59.
 *   - An output may coincide exactly (same pointer, same ld) with an input
 *     of the same type (y with x; dx with x or dy); any other overlap of an
 *     output with an input or another output returns MESWISH_EALIAS.
 *     Interleaved rows that do not touch (two column ranges of one matrix)
 *     do not overlap.
 *   - NaN or infinities in a row make that row's outputs, and dweight,
 *     NaN where the formulas do.
 */
#ifndef LAYER_NORM_H
#define LAYER_NORM_H

#include <stddef.h>

#include "meswish.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward.  weight, bias: n values of param_dtype, or NULL (weight 1,
 * bias 0).  mean, rstd: `rows` binary32 values each, written; either may be
 * NULL (inference).  eps: finite, >= 0.  rows == 0 or n == 0 is a no-op.
 */
int layer_norm_fwd(const void *x, size_t ldx, const void *weight, const void *bias, size_t rows,
                   size_t n, float eps, void *y, size_t ldy, float *mean, float *rstd, int dtype,
                   int param_dtype, void *stream);

/* Bytes of workspace layer_norm_bwd needs when dweight or dbias is asked
 * for (0 otherwise is accepted); 0 if the sizes are out of range. */
size_t layer_norm_workspace_bytes(size_t rows, size_t n);

/*
 * Backward.  mean, rstd: as layer_norm_fwd wrote them.  weight: as in the
 * forward, or NULL.  dweight, dbias: n values of param_dtype, overwritten;
 * either may be NULL (not computed).  workspace: at least
 * layer_norm_workspace_bytes(rows, n) bytes, 4-byte aligned, overwritten;
 * may be NULL if neither dweight nor dbias is asked for.  rows == 0 writes
 * zeros to dweight and dbias; n == 0 is a no-op.
 */
int layer_norm_bwd(const void *x, size_t ldx, const void *dy, size_t lddy, const float *mean,
                   const float *rstd, const void *weight, size_t rows, size_t n, void *dx,
                   size_t lddx, void *dweight, void *dbias, void *workspace,
                   size_t workspace_bytes, int dtype, int param_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_NORM_H */
