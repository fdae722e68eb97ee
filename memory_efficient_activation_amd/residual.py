"""The border between transformer blocks on libmeswish (include/residual_norm.h).

A block's output z enters the residual stream x, with the norms on either side
of the border, in one pass over the rows:

    p = Norm(z) or z                    (post)
    y = skip x + scale gate * p
    o = Norm(y), the next block's input (pre)

A norm is layer normalization, or with ``center`` False the same without the
mean (v / sqrt(mean(v^2) + eps)).  The gate is a vector over the last dimension,
one for all rows or one for each index of x's leading dimensions.  In the manner
of the memory-efficient activations the backward keeps the stream y (which the
next block reads anyway), z, and two values a row and norm.

* ``residual_norm_fwd(x, z, gate, post, pre)`` -> (y, o, RowStats);
* ``residual_norm_bwd(y, z, dy, do, stats, gate, post, pre)`` -> ResidualNormGrads;
* ``ResidualNormFn`` / ``ResidualNorm`` -- an autograd function and module.

Types: x and y float32 or bfloat16; z and o the same, or bfloat16 beside a
float32 stream; weights, biases and gate float32 or bfloat16, all of one type.
Rows at a constant distance are read in place.  Tensor-level functions only
check and marshal arguments; there is no CPU path.  Gradients cannot be
differentiated again (an attempt raises).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch
import torch.nn as nn

from . import _lib
from ._autograd import first_order
from .dense import EPS, SharedBuffer
from .functional import _DTYPES, _dtype_code, _require_device
from .norm import _param, as_rows, launch, library

# A norm's (weight, bias); either may be None: ones, zeros.
Affine = "tuple[torch.Tensor | None, torch.Tensor | None]"


class RowStats(NamedTuple):
    """float32 values of every row; None where a norm is absent, and the means
    where they are not taken off."""
    post_mean: torch.Tensor | None
    post_rstd: torch.Tensor | None
    pre_mean: torch.Tensor | None
    pre_rstd: torch.Tensor | None


class ResidualNormGrads(NamedTuple):
    """None where there is no such parameter, or it is not needed."""
    dx: torch.Tensor
    dz: torch.Tensor
    dgate: torch.Tensor | None
    dpost_weight: torch.Tensor | None
    dpost_bias: torch.Tensor | None
    dpre_weight: torch.Tensor | None
    dpre_bias: torch.Tensor | None


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _branch(t: torch.Tensor, x: torch.Tensor, name: str) -> int:
    """The type code of a tensor [like x] on a block's side of the border."""
    if not t.is_cuda:
        _require_device(t, name)
    if t.get_device() != x.get_device():
        raise ValueError(f"the stream and {name} are on different devices")
    if t.shape != x.shape:
        raise ValueError(f"the stream and {name} have different shapes ({tuple(x.shape)}, "
                         f"{tuple(t.shape)})")
    if t.dtype is not x.dtype and not (x.dtype is torch.float32 and t.dtype is torch.bfloat16):
        raise TypeError(f"{name} must have the stream's dtype {x.dtype}, or bfloat16 beside a "
                        f"float32 stream; got {t.dtype}")
    return _DTYPES[t.dtype]


def _gates(gate: torch.Tensor, x: torch.Tensor) -> int:
    """Rows of the gate: its shape is x's first dimensions and the last."""
    lead = gate.dim() - 1
    if gate.dtype not in _DTYPES:
        raise TypeError(f"gate must be float32 or bfloat16, got {gate.dtype}")
    if not 0 <= lead < x.dim() or gate.shape != (*x.shape[:lead], x.shape[-1]):
        raise ValueError(f"gate must have the stream's first dimensions and its last "
                         f"({tuple(x.shape)}), got {tuple(gate.shape)}")
    if not gate.is_contiguous() or gate.get_device() != x.get_device():
        raise ValueError(f"gate must be contiguous and on {x.device}")
    gates = 1
    for s in gate.shape[:-1]:
        gates *= s
    return gates


def _op(x, rows, n, code, branch, gate, post, pre, skip, scale, center, eps):
    """(the call's description, the parameters' dtype or None)."""
    if post is None and pre is None:
        raise ValueError("at least one of post and pre must be given")
    qw, qb = post if post is not None else (None, None)
    nw, nb = pre if pre is not None else (None, None)
    dtype = None
    for p in (gate, qw, qb, nw, nb):
        if p is None:
            continue
        if dtype is None:
            dtype = p.dtype
        elif p.dtype is not dtype:
            raise TypeError(f"weights, biases and gate have different dtypes ({dtype}, {p.dtype})")
    gates = 1 if gate is None else _gates(gate, x)
    ptrs = (_param(qw, n, x, "post's weight"), _param(qb, n, x, "post's bias"),
            _param(nw, n, x, "pre's weight"), _param(nb, n, x, "pre's bias"))
    # (A gate of no rows, [0, n], beside no rows of x.)
    return _lib.ResidualNormOp(rows, n, gates or 1, _ptr(gate) if gates else None, *ptrs, skip,
                               scale, eps, post is not None, pre is not None, bool(center), code,
                               branch, _DTYPES[dtype] if dtype is not None else _lib.F32), dtype


def residual_norm_fwd(x: torch.Tensor, z: torch.Tensor, gate: torch.Tensor | None = None,
                      post: Affine | None = None, pre: Affine | None = None, scale: float = 1.0,
                      skip: float = 1.0, center: bool = True, eps: float = EPS
                      ) -> tuple[torch.Tensor, torch.Tensor | None, RowStats]:
    """(y, o, statistics): y = skip x + scale gate * p with p = Norm(z) if
    ``post`` is given (z otherwise), o = Norm(y) if ``pre`` is given (None
    otherwise).  ``post`` and ``pre``: (weight, bias), either of which may be
    None; at least one norm is given.  y has x's type, o has z's."""
    code = _dtype_code(x)
    x, rows, n, ldx = as_rows(x, "x")
    branch = _branch(z, x, "z")
    z, _, _, ldz = as_rows(z, "z")
    op, _ = _op(x, rows, n, code, branch, gate, post, pre, scale=scale, skip=skip, center=center,
                eps=eps)
    device, lead = x.device, x.shape[:-1]
    y = torch.empty(x.shape, dtype=x.dtype, device=device)
    o = None if pre is None else torch.empty(x.shape, dtype=z.dtype, device=device)
    used = (post is not None and center, post is not None, pre is not None and center,
            pre is not None)
    planes = iter(torch.empty((sum(used), *lead), dtype=torch.float32, device=device).unbind(0))
    stats = RowStats(*(next(planes) if u else None for u in used))
    launch("residual_norm_fwd", "residual_norm_fwd", device, ctypes.byref(op), x.data_ptr(), ldx,
           z.data_ptr(), ldz, y.data_ptr(), n, _ptr(o), n, *map(_ptr, stats))
    return y, o, stats


def residual_norm_bwd(y: torch.Tensor, z: torch.Tensor, dy: torch.Tensor | None,
                      do: torch.Tensor | None, stats: RowStats, gate: torch.Tensor | None = None,
                      post: Affine | None = None, pre: Affine | None = None, scale: float = 1.0,
                      skip: float = 1.0, center: bool = True, need_params: bool = True,
                      shared: SharedBuffer | None = None) -> ResidualNormGrads:
    """The gradients from y, z, the statistics the forward returned, dy = dL/dy
    (None: zeros) and do = dL/do (with ``pre``).  Those of the parameters and of
    the gate have the parameters' type; with ``need_params`` False they are None.
    ``shared`` lends the workspace."""
    code = _dtype_code(y)
    y, rows, n, ldy = as_rows(y, "y")
    branch = _branch(z, y, "z")
    z, _, _, ldz = as_rows(z, "z")
    op, pdtype = _op(y, rows, n, code, branch, gate, post, pre, scale=scale, skip=skip,
                     center=center, eps=0.0)
    device, lead = y.device, y.shape[:-1]
    lddy = lddo = 0
    if dy is not None:
        if not dy.is_cuda:
            _require_device(dy, "dy")
        if dy.shape != y.shape or dy.dtype is not y.dtype or dy.device != device:
            raise ValueError(f"dy must be a {y.dtype} tensor of shape {tuple(y.shape)} on {device}")
        dy, _, _, lddy = as_rows(dy, "dy")
    if (do is None) != (pre is None):
        raise ValueError("do must be given with pre, and only with it")
    if do is not None:
        if not do.is_cuda:
            _require_device(do, "do")
        if do.shape != y.shape or do.dtype is not z.dtype or do.device != device:
            raise ValueError(f"do must be a {z.dtype} tensor of shape {tuple(y.shape)} on {device}")
        do, _, _, lddo = as_rows(do, "do")
    used = (post is not None and center, post is not None, pre is not None and center,
            pre is not None)
    for name, t, u in zip(RowStats._fields, stats, used):
        if u and (t is None or t.dtype is not torch.float32 or t.shape != lead
                  or t.device != device or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(lead)} "
                             f"on {device}")
    given = [(post or (None, None))[0], (post or (None, None))[1], (pre or (None, None))[0],
             (pre or (None, None))[1]]
    dgate, dparams, ws, nbytes = None, [None] * 4, None, 0
    if need_params:
        if gate is not None:
            dgate = torch.empty(gate.shape, dtype=pdtype, device=device)
        count = sum(p is not None for p in given)
        if count:
            vectors = iter(torch.empty((count, n), dtype=pdtype, device=device).unbind(0))
            dparams = [None if p is None else next(vectors) for p in given]
    dx = torch.empty(y.shape, dtype=y.dtype, device=device)
    dz = torch.empty(y.shape, dtype=z.dtype, device=device)
    nbytes = library().residual_norm_workspace_bytes(rows, n, op.gates if op.gate else 1)
    if nbytes:
        ws = (shared or SharedBuffer()).workspace(nbytes, device)
    launch("residual_norm_bwd", "residual_norm_bwd", device, ctypes.byref(op), y.data_ptr(), ldy,
           z.data_ptr(), ldz, _ptr(dy), lddy, _ptr(do), lddo,
           *(_ptr(t) if u else None for t, u in zip(stats, used)), dx.data_ptr(), n, dz.data_ptr(),
           n, _ptr(dgate) if op.gate else None, *map(_ptr, dparams), _ptr(ws), nbytes)
    return ResidualNormGrads(dx, dz, dgate, *dparams)


class ResidualNormFn(torch.autograd.Function):
    """(y, o) keeping y, z and the rows' statistics; y alone without ``pre``.
    post, pre: whether there is such a norm (its weight and bias may be None)."""

    @staticmethod
    def forward(ctx, x, z, gate, post_weight, post_bias, pre_weight, pre_bias, post, pre, scale,
                skip, center, eps, shared):
        ctx.set_materialize_grads(False)
        y, o, stats = residual_norm_fwd(
            x, z, gate, (post_weight, post_bias) if post else None,
            (pre_weight, pre_bias) if pre else None, scale, skip, center, eps)
        ctx.save_for_backward(y, z, gate, post_weight, post_bias, pre_weight, pre_bias, *stats)
        ctx.args = post, pre, scale, skip, center, shared
        return (y, o) if pre else y

    @staticmethod
    @first_order
    def backward(ctx, dy, do=None):
        y, z, gate, qw, qb, nw, nb, *stats = ctx.saved_tensors
        post, pre, scale, skip, center, shared = ctx.args
        need = ctx.needs_input_grad
        if pre and do is None:
            do = torch.zeros_like(z)
        g = residual_norm_bwd(y, z, dy, do, RowStats(*stats), gate, (qw, qb) if post else None,
                              (nw, nb) if pre else None, scale, skip, center, any(need[2:7]),
                              shared)
        return (*(v if n else None for v, n in zip(g, need)), *[None] * 7)


class ResidualNorm(nn.Module):
    """forward(x, z) -> (y, o), or y without ``pre``: the border behind a block.

    ``post``, ``pre``: whether z, and the sum, are normalized, each with a weight
    and, if ``center`` and ``bias``, a bias.  ``gate``: the initial value of a
    learned gate over the last dimension, or None for none."""

    def __init__(self, n: int, post: bool = True, pre: bool = True, gate: float | None = None,
                 scale: float = 1.0, skip: float = 1.0, center: bool = True, bias: bool = True,
                 eps: float = EPS, shared: SharedBuffer | None = None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        if not (post or pre):
            raise ValueError("at least one of post and pre must be set")
        biases = bias and center
        self.gate = None if gate is None else nn.Parameter(torch.full((n,), gate, dtype=dtype))
        for name, on in (("post", post), ("pre", pre)):
            self.register_parameter(f"{name}_weight",
                                    nn.Parameter(torch.ones(n, dtype=dtype)) if on else None)
            self.register_parameter(f"{name}_bias", nn.Parameter(torch.zeros(n, dtype=dtype))
                                    if on and biases else None)
        self.post, self.pre, self.scale, self.skip = post, pre, float(scale), float(skip)
        self.center, self.eps, self.shared = center, float(eps), shared

    def forward(self, x: torch.Tensor, z: torch.Tensor):
        return ResidualNormFn.apply(x, z, self.gate, self.post_weight, self.post_bias,
                                    self.pre_weight, self.pre_bias, self.post, self.pre,
                                    self.scale, self.skip, self.center, self.eps, self.shared)

    def extra_repr(self) -> str:
        return (f"post={self.post}, pre={self.pre}, gate={self.gate is not None}, "
                f"scale={self.scale}, skip={self.skip}, center={self.center}, eps={self.eps}")
