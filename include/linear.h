/*
 * linear.h -- C ABI of libmeswish's matrix product with its epilogue for AMD
 * Instinct MI355X (gfx950).
 *
 * With x [tokens, dim], W [units, dim], and (each optional) a bias b [units],
 * an activation f of meswish_act and a residual r [tokens, units]:
 *
 *     z = x W^T + b                                [tokens, units]
 *     y = r + f(z)                                           (forward)
 *
 *     dz = dy f'(z)
 *     dx = dz W                                     [tokens, dim]
 *     dW = dz^T x                                   [units, dim]
 *     db = sum over tokens of dz                    [units]  (backward)
 *
 * (dr = dy.)  In the manner of the memory-efficient activations nothing of the
 * forward is kept but x: z never reaches memory in the forward, and the
 * backward computes it again (not without an activation: dz = dy there).
 *
 * Conventions (as in meswish.h): device pointers owned by the caller, no
 * allocation or synchronisation, asynchronous on `stream` (a hipStream_t,
 * NULL = default stream), status codes from meswish_status, nothing
 * launched on an error.
 *   - dtype: MESWISH_F32 or MESWISH_BF16 for every matrix and vector of a call.
 *     Products accumulate in binary32, and z stays binary32 through f, the
 *     bias and the residual.  f and f' are evaluated on it to 1e-5 in binary32
 *     calls, and to 2^-14 in bfloat16 calls (the activations' shorter paths;
 *     the rounding of the result is 2^-9 to 2^-8 of it).  bfloat16 calls round
 *     dz to bfloat16 for the two products that use it (the matrix cores' operand
 *     type; without an activation dz is dy itself); db sums it before.  Every
 *     output is rounded once, to nearest even.
 *   - ld*: elements between the starts of consecutive rows, at least the
 *     row's length and at most LINEAR_MAX_LD; rows are contiguous.  Element
 *     alignment is required.  Rows that do not start on 16-byte boundaries
 *     (pointer, ld and the row's length multiples of 16 bytes) are first copied
 *     to padded ones in the workspace where a product over tiles reads them:
 *     x and w together, and in the backward without an activation dy.
 *   - act, param: as meswish_act_fwd, or LINEAR_IDENTITY for none.
 *   - Results are deterministic: sums have a fixed order, no atomics.  (In binary32
 *     the order of dx's and dw's may depend on whether the other is asked for.)
 *   - Limits: tokens < 2^30; dim, units <= LINEAR_MAX_LD.
 *   - An output may not overlap an input, another output or the workspace
 *     (MESWISH_EALIAS; y may not be r either); column ranges of one matrix do
 *     not overlap.
 *   - No dimension need be positive: a sum over nothing is zero.
 */
#ifndef LINEAR_H
#define LINEAR_H

#include <stddef.h>

#include "meswish.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LINEAR_MAX_LD 2097152
/* No activation: f(z) = z. */
#define LINEAR_IDENTITY (-1)
/* Which rows are aligned, as above. */
#define LINEAR_ALIGNED_XW 1 /* those of x and w */
#define LINEAR_ALIGNED_DY 2 /* those of dy */

/* Bytes of workspace linear_fwd (backward == 0) or linear_bwd (backward != 0)
 * needs; 0 where it needs none or an argument is out of range.  aligned: a sum
 * of LINEAR_ALIGNED_* (0 gives a size that serves any rows; a row length that
 * is not a multiple of 16 bytes counts as not aligned). */
size_t linear_workspace_bytes(size_t tokens, size_t dim, size_t units, int act, int dtype,
                              int backward, int aligned);

/* y [tokens, units].  bias and residual may be NULL.  workspace: 16-byte
 * aligned, at least linear_workspace_bytes(..., 0, aligned) bytes (NULL where
 * that is 0). */
int linear_fwd(int act, float param, const void *x, size_t ldx, const void *w, size_t ldw,
               const void *bias, const void *residual, size_t ldr, size_t tokens, size_t dim,
               size_t units, void *y, size_t ldy, void *workspace, size_t workspace_bytes, int dtype,
               void *stream);

/* dx [tokens, dim], dw [units, dim] and dbias [units] (overwritten, not added
 * to) from x, w, bias (NULL where the forward had none) and dy [tokens, units].
 * Any of the three may be NULL: what is NULL is not computed.  x may be NULL
 * where nothing reads it (no activation, and dw NULL).  workspace: 16-byte
 * aligned, at least linear_workspace_bytes(..., 1, aligned) bytes. */
int linear_bwd(int act, float param, const void *x, size_t ldx, const void *w, size_t ldw,
               const void *bias, const void *dy, size_t lddy, size_t tokens, size_t dim,
               size_t units, void *dx, size_t lddx, void *dw, size_t lddw, void *dbias,
               void *workspace, size_t workspace_bytes, int dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_H */
