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
next block reads anyway; with ``pre``), z (with ``post`` or a learned gate), and two
values a row and norm.

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
    shape, lead = gate.shape, gate.dim() - 1
    if gate.dtype not in _DTYPES:
        raise TypeError(f"gate must be float32 or bfloat16, got {gate.dtype}")
    if not 0 <= lead < x.dim() or shape[lead] != x.shape[-1] or shape[:lead] != x.shape[:lead]:
        raise ValueError(f"gate must have the stream's first dimensions and its last "
                         f"({tuple(x.shape)}), got {tuple(shape)}")
    if not gate.is_contiguous() or gate.get_device() != x.get_device():
        raise ValueError(f"gate must be contiguous and on {x.device}")
    gates = 1
    for s in shape[:lead]:
        gates *= s
    return gates


def _same_dtype(dtype: torch.dtype | None, p: torch.Tensor) -> torch.dtype:
    if dtype is not None and p.dtype is not dtype:
        raise TypeError(f"weights, biases and gate have different dtypes ({dtype}, {p.dtype})")
    return p.dtype


def _norm_ptrs(norm, dtype, n, x, name):
    """(weight's address, bias's, the parameters' dtype so far); 0: none."""
    w, b = norm
    wp = bp = 0
    if w is not None:
        dtype = _same_dtype(dtype, w)
        wp = _param(w, n, x, name + "'s weight")
    if b is not None:
        dtype = _same_dtype(dtype, b)
        bp = _param(b, n, x, name + "'s bias")
    return wp, bp, dtype


def _op(x, rows, n, code, branch, gate, post, pre, skip, scale, center, eps):
    """(the call's packed description, the parameters' dtype or None, the gate's
    rows, whether it is used)."""
    if post is None and pre is None:
        raise ValueError("at least one of post and pre must be given")
    dtype, gates, gp = None, 1, 0
    if gate is not None:
        dtype, gates = gate.dtype, _gates(gate, x)
        if gates:
            gp = gate.data_ptr()
        else:  # a gate of no rows, [0, n], beside no rows of x
            gates = 1
    qw = qb = nw = nb = 0
    if post is not None:
        qw, qb, dtype = _norm_ptrs(post, dtype, n, x, "post")
    if pre is not None:
        nw, nb, dtype = _norm_ptrs(pre, dtype, n, x, "pre")
    return (_lib.RESIDUAL_NORM_OP.pack(rows, n, gates, gp, qw, qb, nw, nb, skip, scale, eps,
                                       post is not None, pre is not None, bool(center), code,
                                       branch, 0 if dtype is None else _DTYPES[dtype]),
            dtype, gates, gp != 0)


def _new_like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t) if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device)


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
    op = _op(x, rows, n, code, branch, gate, post, pre, skip, scale, center, eps)[0]
    device, lead = x.device, x.shape[:-1]
    y = _new_like(x)
    o = op_ = qm = qr = nm = nr = None
    k = 2 if center else 1
    both = post is not None and pre is not None
    planes = torch.empty((2 * k if both else k, *lead), dtype=torch.float32, device=device).unbind(0)
    if pre is not None:
        o = _new_like(z)
        op_, nr = o.data_ptr(), planes[-1]
        nm = planes[-2] if center else None
    if post is not None:
        qr, qm = planes[k - 1], planes[0] if center else None
    launch("residual_norm_fwd", "residual_norm_fwd", device, op, x.data_ptr(), ldx, z.data_ptr(),
           ldz, y.data_ptr(), n, op_, n, _ptr(qm), _ptr(qr), _ptr(nm), _ptr(nr))
    return y, o, RowStats(qm, qr, nm, nr)


def _upstream(t: torch.Tensor, like: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    if not t.is_cuda:
        _require_device(t, name)
    if t.shape != like.shape or t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a {like.dtype} tensor of shape {tuple(like.shape)} on "
                         f"{like.device}")
    t, _, _, ld = as_rows(t, name)
    return t, ld


def _stat(t: torch.Tensor | None, lead, y: torch.Tensor, name: str) -> int:
    if t is None or t.dtype is not torch.float32 or t.shape != lead or not t.is_contiguous() \
            or t.get_device() != y.get_device():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(lead)} on "
                         f"{y.device}")
    return t.data_ptr()


def residual_norm_bwd(y: torch.Tensor, z: torch.Tensor, dy: torch.Tensor | None,
                      do: torch.Tensor | None, stats: RowStats, gate: torch.Tensor | None = None,
                      post: Affine | None = None, pre: Affine | None = None, scale: float = 1.0,
                      skip: float = 1.0, center: bool = True,
                      need_params: bool | tuple[bool, ...] = True,
                      shared: SharedBuffer | None = None) -> ResidualNormGrads:
    """The gradients from y, z, the statistics the forward returned, dy = dL/dy
    (None, with ``pre``: zeros) and do = dL/do (with ``pre``).  Those of the
    parameters and of the gate have the parameters' type.  ``need_params``: whether
    they are computed, or for each of (gate, post's weight, its bias, pre's weight,
    its bias); what is not needed is None.  y is read only with ``pre``, z only with
    ``post`` or for the gate's gradient; elsewhere any tensors like them will do.
    ``shared`` lends the workspace."""
    code = _dtype_code(y)
    y, rows, n, ldy = as_rows(y, "y")
    branch = _branch(z, y, "z")
    z, _, _, ldz = as_rows(z, "z")
    op, pdtype, gates, gated = _op(y, rows, n, code, branch, gate, post, pre, skip, scale, center,
                                   0.0)
    device, lead = y.device, y.shape[:-1]
    dyp = dop = qm = qr = nm = nr = None
    lddy = lddo = 0
    if dy is not None:
        dy, lddy = _upstream(dy, y, "dy")
        dyp = dy.data_ptr()
    elif pre is None:
        raise ValueError("dy must be given without pre")
    if (do is None) != (pre is None):
        raise ValueError("do must be given with pre, and only with it")
    if pre is not None:
        do, lddo = _upstream(do, z, "do")
        dop = do.data_ptr()
        nm = _stat(stats[2], lead, y, "pre_mean") if center else None
        nr = _stat(stats[3], lead, y, "pre_rstd")
    if post is not None:
        qm = _stat(stats[0], lead, y, "post_mean") if center else None
        qr = _stat(stats[1], lead, y, "post_rstd")
    given = (*(post or (None, None)), *(pre or (None, None)))
    dgate, grads, ptrs = None, [None] * 4, [None] * 4
    if need_params:
        need = need_params if isinstance(need_params, tuple) else (True,) * 5
        if len(need) != 5:
            raise ValueError(f"need_params names five gradients, got {len(need)}")
        if gate is not None and need[0]:
            dgate = torch.empty_like(gate)
        wanted = [i for i, p in enumerate(given) if p is not None and need[i + 1]]
        if wanted:
            vectors = torch.empty((len(wanted), n), dtype=pdtype, device=device).unbind(0)
            for i, g in zip(wanted, vectors):
                grads[i] = g
                ptrs[i] = g.data_ptr()
    dx, dz = _new_like(y), _new_like(z)
    nbytes = library().residual_norm_workspace_bytes(rows, n, gates)
    ws = (shared or SharedBuffer()).workspace(nbytes, device)
    launch("residual_norm_bwd", "residual_norm_bwd", device, op, y.data_ptr(), ldy, z.data_ptr(),
           ldz, dyp, lddy, dop, lddo, qm, qr, nm, nr, dx.data_ptr(), n, dz.data_ptr(), n,
           dgate.data_ptr() if gated and dgate is not None else None, *ptrs, ws.data_ptr(), nbytes)
    return ResidualNormGrads(dx, dz, dgate, *grads)


class ResidualNormFn(torch.autograd.Function):
    """(y, o) keeping what the backward reads: y under the norm behind it, z under the
    norm before it or for the gate's gradient, and the rows' statistics; y alone
    without ``pre``.  post, pre: whether there is such a norm (its weight and bias may
    be None)."""

    @staticmethod
    def forward(ctx, x, z, gate, post_weight, post_bias, pre_weight, pre_bias, post, pre, scale,
                skip, center, eps, shared):
        ctx.set_materialize_grads(False)
        y, o, stats = residual_norm_fwd(
            x, z, gate, (post_weight, post_bias) if post else None,
            (pre_weight, pre_bias) if pre else None, scale, skip, center, eps)
        of_gate = gate is not None and ctx.needs_input_grad[2]
        ctx.save_for_backward(y if pre else None, z if post or of_gate else None, gate, post_weight,
                              post_bias, pre_weight, pre_bias, *stats)
        ctx.args = post, pre, scale, skip, center, shared, x.dtype, z.dtype
        return (y, o) if pre else y

    @staticmethod
    @first_order
    def backward(ctx, dy, do=None):
        y, z, gate, qw, qb, nw, nb, *stats = ctx.saved_tensors
        post, pre, scale, skip, center, shared, stream, branch = ctx.args
        need = ctx.needs_input_grad
        if pre and do is None:
            do = torch.zeros(y.shape, dtype=branch, device=y.device)
        if not pre and dy is None:
            dy = torch.zeros(z.shape, dtype=stream, device=z.device)
        # What was not kept is not read: its gradient is a tensor like it.
        if y is None:
            y = dy = dy.contiguous()
        if z is None:
            z = do = do.contiguous()
        g = residual_norm_bwd(y, z, dy, do, RowStats(*stats), gate, (qw, qb) if post else None,
                              (nw, nb) if pre else None, scale, skip, center,
                              any(need[2:7]) and need[2:7], shared)
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
