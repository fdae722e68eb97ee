/*
 * gated_ffn.h -- C ABI of libmeswish's gated feed-forward unit for AMD
 * Instinct MI355X (gfx950).
 *
 * With x [tokens, dim], Wg and Wu [hidden, dim] and an activation f of
 * meswish_act (Swish gives the unit usually called SwiGLU, the GELUs GEGLU,
 * sigmoid GLU, ReLU ReGLU):
 *
 *     g = x Wg^T,  u = x Wu^T                       [tokens, hidden]
 *     h = f(g) * u                                              (forward)
 *
 *     dg = dh * u * f'(g),  du = dh * f(g)
 *     dx  = dg Wg + du Wu                           [tokens, dim]
 *     dWg = dg^T x,  dWu = du^T x                   [hidden, dim] (backward)
 *
 * In the manner of the memory-efficient activations nothing of the forward
 * is kept but x: neither g, u nor f(g) reaches memory in the forward, and
 * the backward computes both projections again.
 *
 * Conventions (as in meswish.h): device pointers owned by the caller, no
 * allocation or synchronisation, asynchronous on `stream` (a hipStream_t,
 * NULL = default stream), status codes from meswish_status, nothing
 * launched on an error.
 *   - dtype: MESWISH_F32 or MESWISH_BF16 for every matrix of a call.
 *     Products accumulate in binary32; g and u stay binary32 through f.
 *     f and f' are evaluated on them to 1e-5 in binary32 calls, and to 2^-14
 *     in bfloat16 calls (the activations' shorter paths; the rounding of the
 *     result is 2^-9 to 2^-8 of it).
 *     bfloat16 calls round dg and du to bfloat16 for the products that use
 *     them (the matrix cores' operand type).  Every output is rounded once,
 *     to nearest even.
 *   - ld*: elements between the starts of consecutive rows, at least the
 *     row's length and at most GATED_FFN_MAX_LD; rows are contiguous.
 *     Element alignment is required.  Where a row of x, wg or wu does not
 *     start on a 16-byte boundary (pointers, ld a multiple of 16 bytes, the
 *     same ld for wg and wu), or dim is not a multiple of 16 bytes, all three
 *     are first copied to padded rows in the workspace (not for the forward
 *     of at most 32 tokens, which takes any rows).
 *   - act, param: as meswish_act_fwd.
 *   - Results are deterministic: sums have a fixed order, no atomics.
 *   - Limits: tokens < 2^30; dim, hidden <= GATED_FFN_MAX_LD.
 *   - An output may not overlap an input, another output or the workspace
 *     (MESWISH_EALIAS); column ranges of one matrix do not overlap.
 *   - No dimension need be positive: a sum over nothing is zero.
 */
#ifndef GATED_FFN_H
#define GATED_FFN_H

#include <stddef.h>

#include "meswish.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GATED_FFN_MAX_LD 2097152

/* Bytes of workspace gated_ffn_fwd (backward == 0) or gated_ffn_bwd
 * (backward != 0) needs; 0 where it needs none or the sizes are out of
 * range.  aligned: whether the rows of x, wg and wu are, as above (0 gives a
 * size that serves any rows; a dim that is not a multiple of 16 bytes counts
 * as 0). */
size_t gated_ffn_workspace_bytes(size_t tokens, size_t dim, size_t hidden, int dtype,
                                 int backward, int aligned);

/* h [tokens, hidden] from x, wg, wu.  workspace: 16-byte aligned, at least
 * gated_ffn_workspace_bytes(..., 0, aligned) bytes (NULL where that is 0). */
int gated_ffn_fwd(int act, float param, const void *x, size_t ldx, const void *wg, size_t ldwg,
                  const void *wu, size_t ldwu, size_t tokens, size_t dim, size_t hidden, void *h,
                  size_t ldh, void *workspace, size_t workspace_bytes, int dtype, void *stream);

/* dx [tokens, dim], dwg and dwu [hidden, dim] (overwritten, not added to)
 * from x, wg, wu and dh [tokens, hidden].  dx may be NULL, and so may dwg
 * and dwu together: what is NULL is not computed.  h: NULL, or [tokens,
 * hidden], where the forward's result is written again (for the gradient
 * of the projection that follows, which then need not keep it either).
 * workspace: 16-byte aligned, at least gated_ffn_workspace_bytes(..., 1,
 * aligned) bytes. */
int gated_ffn_bwd(int act, float param, const void *x, size_t ldx, const void *wg, size_t ldwg,
                  const void *wu, size_t ldwu, const void *dh, size_t lddh, size_t tokens,
                  size_t dim, size_t hidden, void *dx, size_t lddx, void *dwg, size_t lddwg,
                  void *dwu, size_t lddwu, void *h, size_t ldh, void *workspace,
                  size_t workspace_bytes, int dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_FFN_H */
