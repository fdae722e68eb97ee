"""Gated feed-forward unit and block on libmeswish (include/gated_ffn.h).

h = f(x Wg^T) * (x Wu^T), f any activation of the family (Swish: the unit
usually called SwiGLU; the GELUs: GEGLU; sigmoid: GLU; ReLU: ReGLU).  One
kernel computes both projections, the activation and the product; in the
manner of the memory-efficient activations the backward keeps x alone and
computes both projections again.

* ``gated_ffn_fwd(x, w_gate, w_up, kind, param)`` -> h;
* ``gated_ffn_bwd(x, w_gate, w_up, dh, kind, param)`` -> (dx, dw_gate,
  dw_up), and h again on request;
* ``GatedFFNFn`` / ``GatedUnit`` -- an autograd function and module;
* ``PreNormGatedFeedForward`` -- the transformer's feed-forward block
  x + W_down h(LN(x)) with the layer normalization of ``norm``, keeping x
  and two values a token for the backward.

Weights are [hidden, dim], as ``torch.nn.Linear`` holds them.  float32 or
bfloat16.  Tensor-level functions only check and marshal arguments; there is
no CPU path.  Gradients cannot be differentiated again (an attempt raises).
The block's last projection is a plain product and PyTorch's: it is the model
around the operators.
"""

from __future__ import annotations

import torch
import torch.nn as nn

from . import _lib
from ._autograd import first_order
from .dense import EPS, SharedBuffer
from .functional import _act_code, _dtype_code, _require_device
from .norm import _out_rows, as_rows, launch, layer_norm_bwd, layer_norm_fwd, library


def _rows(t: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    """t and the distance of its rows, copied where no one distance serves or
    the library does not take it (one token of each long sequence, say)."""
    t, _, n, ld = as_rows(t, name)
    if ld > _lib.GATED_FFN_MAX_LD and ld > n:
        t, ld = t.contiguous(), n
    return t, ld


def _weight(x: torch.Tensor, w: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    """w and its row distance, checked against x."""
    if not w.is_cuda:
        _require_device(w, name)
    if w.get_device() != x.get_device():
        raise ValueError(f"x and {name} are on different devices")
    if w.dtype is not x.dtype:
        raise TypeError(f"x and {name} have different dtypes ({x.dtype}, {w.dtype})")
    if w.dim() != 2 or w.shape[1] != x.shape[-1]:
        raise ValueError(f"{name} must be [hidden, {x.shape[-1]}], got {tuple(w.shape)}")
    return _rows(w, name)


def _weights(x, w_gate, w_up):
    if w_gate.shape != w_up.shape:
        raise ValueError(f"w_gate and w_up have different shapes ({tuple(w_gate.shape)}, "
                         f"{tuple(w_up.shape)})")
    return _weight(x, w_gate, "w_gate"), _weight(x, w_up, "w_up")


def _param_value(kind: str, param: float | None) -> float:
    return _lib.DEFAULT_PARAM.get(kind, 0.0) if param is None else float(param)


def _tokens(x: torch.Tensor) -> int:
    n = 1
    for s in x.shape[:-1]:
        n *= s
    return n


def _aligned(x, ldx, wg, ldg, wu, ldu, dim) -> bool:
    """Whether the rows of all three start on 16-byte boundaries."""
    per = 16 // x.element_size()
    return not ((x.data_ptr() | wg.data_ptr() | wu.data_ptr()) % 16 or (ldx | ldg | dim) % per
                or ldg != ldu)


def _workspace(tokens, dim, hidden, code, backward, aligned, device, shared):
    nbytes = library().gated_ffn_workspace_bytes(tokens, dim, hidden, code, backward, aligned)
    if nbytes == 0:
        return None, 0
    ws = (shared or SharedBuffer()).workspace(nbytes, device)
    return ws, nbytes


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def gated_ffn_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, kind: str = "swish",
                  param: float | None = None, out: torch.Tensor | None = None,
                  shared: SharedBuffer | None = None) -> torch.Tensor:
    """h = f(x w_gate^T) * (x w_up^T), [..., hidden].  ``shared`` lends its
    workspace."""
    act = _act_code(kind)
    code = _dtype_code(x)
    x, ldx = _rows(x, "x")
    dim = x.shape[-1]
    (wg, ldg), (wu, ldu) = _weights(x, w_gate, w_up)
    tokens, hidden = _tokens(x), w_gate.shape[0]
    shape = (*x.shape[:-1], hidden)
    if out is None:
        h, ldh = torch.empty(shape, dtype=x.dtype, device=x.device), hidden
    else:
        if out.shape != shape or out.dtype != x.dtype or out.device != x.device:
            raise ValueError(f"out must be a {x.dtype} tensor of shape {shape} on {x.device}")
        h, ldh = _out_rows(out, out, "out")
        if ldh > _lib.GATED_FFN_MAX_LD and ldh > hidden:
            raise ValueError(f"the rows of out are {ldh} elements apart, more than "
                             f"{_lib.GATED_FFN_MAX_LD}")
    device = x.device
    ws, nbytes = _workspace(tokens, dim, hidden, code, 0,
                            _aligned(x, ldx, wg, ldg, wu, ldu, dim), device, shared)
    launch("gated_ffn_fwd", f"gated_ffn_fwd({kind})", device, act, _param_value(kind, param),
           x.data_ptr(), ldx, wg.data_ptr(), ldg, wu.data_ptr(), ldu, tokens, dim, hidden,
           h.data_ptr(), ldh, _ptr(ws), nbytes, code)
    return h


def gated_ffn_bwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, dh: torch.Tensor,
                  kind: str = "swish", param: float | None = None, need_x: bool = True,
                  need_weights: bool = True, need_h: bool = False,
                  shared: SharedBuffer | None = None) -> tuple[torch.Tensor | None, ...]:
    """(dx, dw_gate, dw_up) from the input, the weights and dh = dL/dh, both
    projections recomputed; with ``need_h`` also h, computed on the way.
    What is not needed is None.  ``shared`` lends its workspace."""
    act = _act_code(kind)
    code = _dtype_code(x)
    if not dh.is_cuda:
        _require_device(dh, "dh")
    x, ldx = _rows(x, "x")
    dim = x.shape[-1]
    (wg, ldg), (wu, ldu) = _weights(x, w_gate, w_up)
    tokens, hidden = _tokens(x), w_gate.shape[0]
    if dh.shape != (*x.shape[:-1], hidden) or dh.dtype != x.dtype or dh.device != x.device:
        raise ValueError(f"dh must be a {x.dtype} tensor of shape {(*x.shape[:-1], hidden)} on "
                         f"{x.device}")
    dh, lddh = _rows(dh, "dh")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_x else None
    dwg = dwu = None
    if need_weights:
        dwg = torch.empty((hidden, dim), dtype=x.dtype, device=x.device)
        dwu = torch.empty((hidden, dim), dtype=x.dtype, device=x.device)
    h = torch.empty(dh.shape, dtype=x.dtype, device=x.device) if need_h else None
    device = x.device
    ws, nbytes = _workspace(tokens, dim, hidden, code, 1,
                            _aligned(x, ldx, wg, ldg, wu, ldu, dim), device, shared)
    launch("gated_ffn_bwd", f"gated_ffn_bwd({kind})", device, act, _param_value(kind, param),
           x.data_ptr(), ldx, wg.data_ptr(), ldg, wu.data_ptr(), ldu, dh.data_ptr(), lddh, tokens,
           dim, hidden, _ptr(dx), dim, _ptr(dwg), dim, _ptr(dwu), dim, _ptr(h), hidden, _ptr(ws),
           nbytes, code)
    return (dx, dwg, dwu, h) if need_h else (dx, dwg, dwu)


class GatedFFNFn(torch.autograd.Function):
    """The gated unit keeping x (and references to the weights)."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, kind, param, shared):
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.kind, ctx.param, ctx.shared = kind, param, shared
        return gated_ffn_fwd(x, w_gate, w_up, kind, param, shared=shared)

    @staticmethod
    @first_order
    def backward(ctx, dh):
        x, w_gate, w_up = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dwg, dwu = gated_ffn_bwd(x, w_gate, w_up, dh, ctx.kind, ctx.param, need[0],
                                     need[1] or need[2], shared=ctx.shared)
        return dx, dwg if need[1] else None, dwu if need[2] else None, None, None, None


class GatedUnit(nn.Module):
    """f(x w_gate^T) * (x w_up^T) over the last dimension (dim -> hidden)."""

    def __init__(self, dim: int, hidden: int, kind: str = "swish", param: float | None = None,
                 shared: SharedBuffer | None = None, dtype: torch.dtype = torch.float32):
        super().__init__()
        _act_code(kind)
        self.w_gate = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.w_up = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.kind, self.param, self.shared = kind, param, shared

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return GatedFFNFn.apply(x, self.w_gate, self.w_up, self.kind, self.param, self.shared)

    def extra_repr(self) -> str:
        hidden, dim = self.w_gate.shape
        return f"{dim}, {hidden}, kind={self.kind}, param={self.param}"


class PreNormGatedFFNFn(torch.autograd.Function):
    """x + h(LN(x)) W_down^T keeping x and the rows' statistics: the
    backward normalizes again and takes h from the unit's backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, w_gate, w_up, w_down, kind, param, eps, shared):
        n, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        h = gated_ffn_fwd(n, w_gate, w_up, kind, param, shared=shared)
        ctx.save_for_backward(x, mean, rstd, weight, bias, w_gate, w_up, w_down)
        ctx.kind, ctx.param, ctx.eps, ctx.shared = kind, param, eps, shared
        return torch.addmm(x.reshape(-1, x.shape[-1]), h.view(-1, h.shape[-1]),
                           w_down.t()).view(x.shape)

    @staticmethod
    @first_order
    def backward(ctx, dy):
        x, mean, rstd, weight, bias, w_gate, w_up, w_down = ctx.saved_tensors
        need = ctx.needs_input_grad  # x, weight, bias, w_gate, w_up, w_down, ...
        need_norm, need_unit = any(need[:3]), need[3] or need[4]
        dy = dy.contiguous()
        dy2 = dy.view(-1, dy.shape[-1])
        n = layer_norm_fwd(x, weight, bias, ctx.eps)[0]
        dx = dw = db = dwg = dwu = dwd = h = None
        if need_norm or need_unit:
            dh = (dy2 @ w_down).view(*x.shape[:-1], w_down.shape[1])
            dn, dwg, dwu, *rest = gated_ffn_bwd(n, w_gate, w_up, dh, ctx.kind, ctx.param, need_norm,
                                                need_unit, need[5], shared=ctx.shared)
            h = rest[0] if need[5] else None
        elif need[5]:
            h = gated_ffn_fwd(n, w_gate, w_up, ctx.kind, ctx.param, shared=ctx.shared)
        if need[5]:
            dwd = dy2.t() @ h.view(-1, h.shape[-1])
        if need_norm:
            dx, dw, db = layer_norm_bwd(x, dn, mean, rstd, weight, need[1] or need[2],
                                        shared=ctx.shared)
            dx = dx.add_(dy) if need[0] else None
        grads = (dx, dw, db, dwg, dwu, dwd)
        return (*(g if wanted else None for g, wanted in zip(grads, need)), None, None, None, None)


class PreNormGatedFeedForward(nn.Module):
    """The transformer's feed-forward block x + W_down h(LN(x)), every
    parameter in ``dtype``.  Blocks may share one SharedBuffer, if their calls
    follow each other on one stream (and come from one thread); without one
    each call has a workspace of its own."""

    def __init__(self, dim: int, hidden: int, kind: str = "swish", param: float | None = None,
                 eps: float = EPS, shared: SharedBuffer | None = None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        _act_code(kind)
        self.weight = nn.Parameter(torch.ones(dim, dtype=dtype))
        self.bias = nn.Parameter(torch.zeros(dim, dtype=dtype))
        self.w_gate = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.w_up = nn.Parameter(torch.randn(hidden, dim, dtype=dtype) * dim ** -0.5)
        self.w_down = nn.Parameter(torch.randn(dim, hidden, dtype=dtype) * hidden ** -0.5)
        self.kind, self.param, self.eps, self.shared = kind, param, float(eps), shared

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return PreNormGatedFFNFn.apply(x, self.weight, self.bias, self.w_gate, self.w_up,
                                       self.w_down, self.kind, self.param, self.eps, self.shared)

    def extra_repr(self) -> str:
        hidden, dim = self.w_gate.shape
        return f"{dim}, {hidden}, kind={self.kind}, param={self.param}, eps={self.eps}"
