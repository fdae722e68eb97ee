"""Feed-forward blocks made of the library's products, norms and borders.

In the manner of the memory-efficient activations each keeps its input and the
rows' statistics, and computes what lies between again in its backward:

* ``PreNormFeedForward`` -- x + W2 f(W1 LN(x) + b1) + b2, the block without a
  gate: two products (include/linear.h), the first with its bias and activation
  in the epilogue, the second with its bias and the residual sum;
* ``GatedFeedForward`` -- W_down (f(n Wg^T) * (n Wu^T)), the gated unit and the
  product behind it, of rows that are normalized already;
* ``GatedFeedForwardStack`` -- such blocks joined by borders
  (include/residual_norm.h): each block's output is normalized, gated and summed
  into the stream, and the sum normalized for the next block, in one pass.

float32 or bfloat16, every parameter in one type.  Modules may share one
SharedBuffer, if their calls follow each other on one stream (and come from one
thread); without one each call has a workspace of its own.
"""

from __future__ import annotations

import torch
import torch.nn as nn

from . import residual
from ._autograd import first_order
from .dense import EPS, SharedBuffer
from .ffn import gated_ffn_bwd, gated_ffn_fwd
from .functional import _act_code
from .linear import linear_bwd, linear_fwd
from .norm import LayerNorm, layer_norm_bwd, layer_norm_fwd
from .residual import ResidualNorm


class PreNormFeedForwardFn(torch.autograd.Function):
    """x + W2 f(W1 LN(x) + b1) + b2 keeping x and the rows' statistics."""

    @staticmethod
    def forward(ctx, x, weight, bias, w1, b1, w2, b2, kind, param, eps, shared):
        n, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        a = linear_fwd(n, w1, b1, None, kind, param, shared=shared)
        ctx.save_for_backward(x, mean, rstd, weight, bias, w1, b1, w2, b2)
        ctx.kind, ctx.param, ctx.eps, ctx.shared = kind, param, eps, shared
        return linear_fwd(a, w2, b2, x, shared=shared)

    @staticmethod
    @first_order
    def backward(ctx, dy):
        x, mean, rstd, weight, bias, w1, b1, w2, b2 = ctx.saved_tensors
        need, shared = ctx.needs_input_grad, ctx.shared  # x, weight, bias, w1, b1, w2, b2, ...
        need_norm, need_first = any(need[:3]), any(need[:5])
        dx = dw = db = dw1 = db1 = dw2 = db2 = None
        n = layer_norm_fwd(x, weight, bias, ctx.eps)[0] if need_first or need[5] else None
        if need_first or need[5] or need[6]:
            a = None  # what f gave: W2's gradient alone reads it
            if need[5]:
                a = linear_fwd(n, w1, b1, None, ctx.kind, ctx.param, shared=shared)
            da, dw2, db2 = linear_bwd(a, w2, dy, None, None, None, need_first, need[5], need[6],
                                      shared=shared)
            del a
        if need_first:
            dn, dw1, db1 = linear_bwd(n, w1, da, b1, ctx.kind, ctx.param, need_norm, need[3],
                                      need[4], shared=shared)
            del da
        if need[0]:
            # The border behind y = x: dy and the norm's share are added in binary32 and
            # rounded once.
            g = residual.residual_norm_bwd(x, dn, dy, dn, residual.RowStats(None, None, mean, rstd),
                                           pre=(weight, bias),
                                           need_params=(False, False, False, need[1], need[2]),
                                           shared=shared)
            dx, dw, db = g.dx, g.dpre_weight, g.dpre_bias
        elif need_norm:  # reads no dy, and writes a map less
            dw, db = layer_norm_bwd(x, dn, mean, rstd, weight, shared=shared)[1:]
        grads = (dx, dw, db, dw1, db1, dw2, db2)
        return (*(g if wanted else None for g, wanted in zip(grads, need)), None, None, None, None)


class PreNormFeedForward(nn.Module):
    """The feed-forward block without a gate, x + W2 f(W1 LN(x) + b1) + b2."""

    def __init__(self, dim: int, hidden: int, kind: str = "gelu", param: float | None = None,
                 bias: bool = True, eps: float = EPS, shared: SharedBuffer | None = None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        _act_code(kind)
        self.weight = nn.Parameter(torch.ones(dim, dtype=dtype))
        self.bias = nn.Parameter(torch.zeros(dim, dtype=dtype))
        self.w1 = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.b1 = nn.Parameter(torch.zeros(hidden, dtype=dtype)) if bias else None
        self.w2 = nn.Parameter(torch.randn(dim, hidden, dtype=dtype) * hidden ** -0.5)
        self.b2 = nn.Parameter(torch.zeros(dim, dtype=dtype)) if bias else None
        self.kind, self.param, self.eps, self.shared = kind, param, float(eps), shared

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return PreNormFeedForwardFn.apply(x, self.weight, self.bias, self.w1, self.b1, self.w2,
                                          self.b2, self.kind, self.param, self.eps, self.shared)

    def extra_repr(self) -> str:
        hidden, dim = self.w1.shape
        return (f"{dim}, {hidden}, kind={self.kind}, param={self.param}, "
                f"bias={self.b1 is not None}, eps={self.eps}")


class GatedFeedForwardFn(torch.autograd.Function):
    """W_down (f(n Wg^T) * (n Wu^T)) keeping n: the product h of the unit comes
    out of the unit's backward again."""

    @staticmethod
    def forward(ctx, n, w_gate, w_up, w_down, kind, param, shared):
        ctx.save_for_backward(n, w_gate, w_up, w_down)
        ctx.kind, ctx.param, ctx.shared = kind, param, shared
        h = gated_ffn_fwd(n, w_gate, w_up, kind, param, shared=shared)
        return linear_fwd(h, w_down, shared=shared)

    @staticmethod
    @first_order
    def backward(ctx, dz):
        n, w_gate, w_up, w_down = ctx.saved_tensors
        need, shared = ctx.needs_input_grad, ctx.shared  # n, w_gate, w_up, w_down, ...
        need_unit = need[1] or need[2]
        dn = dwg = dwu = dwd = h = None
        if need[0] or need_unit:
            dh = linear_bwd(None, w_down, dz, need_weight=False, shared=shared)[0]
            dn, dwg, dwu, *rest = gated_ffn_bwd(n, w_gate, w_up, dh, ctx.kind, ctx.param, need[0],
                                                need_unit, need[3], shared=shared)
            h = rest[0] if need[3] else None
        elif need[3]:
            h = gated_ffn_fwd(n, w_gate, w_up, ctx.kind, ctx.param, shared=shared)
        if need[3]:
            dwd = linear_bwd(h, w_down, dz, need_x=False, shared=shared)[1]
        return dn, dwg if need[1] else None, dwu if need[2] else None, dwd, None, None, None


class GatedFeedForward(nn.Module):
    """W_down (f(n w_gate^T) * (n w_up^T)) over the last dimension."""

    def __init__(self, dim: int, hidden: int, kind: str = "swish", param: float | None = None,
                 shared: SharedBuffer | None = None, dtype: torch.dtype = torch.float32):
        super().__init__()
        _act_code(kind)
        self.w_gate = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.w_up = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.w_down = nn.Parameter(torch.randn(dim, hidden, dtype=dtype) * hidden ** -0.5)
        self.kind, self.param, self.shared = kind, param, shared

    def forward(self, n: torch.Tensor) -> torch.Tensor:
        return GatedFeedForwardFn.apply(n, self.w_gate, self.w_up, self.w_down, self.kind,
                                        self.param, self.shared)

    def extra_repr(self) -> str:
        hidden, dim = self.w_gate.shape
        return f"{dim}, {hidden}, kind={self.kind}, param={self.param}"


class GatedFeedForwardStack(nn.Module):
    """forward(x) -> LN(y) of the last block's stream y, from

        n = LN(x), then block by block  z = block(n),
        x = x + scale gate * LN(z) (or z without ``post``),  n = LN(x).

    ``gate``: the learned gates' initial value, or None for none."""

    def __init__(self, dim: int, hidden: int, blocks: int, kind: str = "swish",
                 param: float | None = None, post: bool = True, gate: float | None = None,
                 scale: float = 1.0, eps: float = EPS, shared: SharedBuffer | None = None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        self.norm = LayerNorm(dim, eps, shared=shared, dtype=dtype)
        self.blocks = nn.ModuleList(GatedFeedForward(dim, hidden, kind, param, shared, dtype)
                                    for _ in range(blocks))
        self.borders = nn.ModuleList(ResidualNorm(dim, post, True, gate, scale, eps=eps,
                                                  shared=shared, dtype=dtype)
                                     for _ in range(blocks))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        n = self.norm(x)
        for block, border in zip(self.blocks, self.borders):
            x, n = border(x, block(n))
        return n
