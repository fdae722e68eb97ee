"""Matrix product with its epilogue on libmeswish (include/linear.h).

y = residual + f(x W^T + bias), f any activation of the family or none, bias and
residual optional.  One kernel computes the product and what follows it; in the
manner of the memory-efficient activations the backward keeps x alone and
computes the product under f' again (without an activation it needs none, nor x
unless the weight has a gradient).

* ``linear_fwd(x, weight, bias, residual, kind, param)`` -> y;
* ``linear_bwd(x, weight, dy, bias, kind, param)`` -> (dx, dweight, dbias);
* ``LinearFn`` / ``Linear`` -- an autograd function and module.

The weight is [units, dim], as ``torch.nn.Linear`` holds it.  float32 or
bfloat16, one type for all tensors of a call.  Tensor-level functions only
check and marshal arguments; there is no CPU path.  Gradients cannot be
differentiated again (an attempt raises).
"""

from __future__ import annotations

import torch
import torch.nn as nn

from . import _lib
from ._autograd import first_order
from .dense import SharedBuffer
from .ffn import _param_value, _ptr, _tokens
from .functional import _act_code, _dtype_code, _require_device
from .norm import _out_rows, as_rows, launch, library


def _code(kind: str | None) -> int:
    return _lib.LINEAR_IDENTITY if kind is None else _act_code(kind)


def _rows(t: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    """t and the distance of its rows, copied where no one distance serves or
    the library does not take it."""
    t, _, n, ld = as_rows(t, name)
    if ld > _lib.LINEAR_MAX_LD and ld > n:
        t, ld = t.contiguous(), n
    return t, ld


def _like(t: torch.Tensor, shape, x: torch.Tensor, name: str) -> None:
    """t is of x's type and device and of the shape."""
    if not t.is_cuda:
        _require_device(t, name)
    if t.get_device() != x.get_device():
        raise ValueError(f"x and {name} are on different devices")
    if t.dtype is not x.dtype:
        raise TypeError(f"x and {name} have different dtypes ({x.dtype}, {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _weight(w: torch.Tensor, x: torch.Tensor, dim: int | None) -> tuple[torch.Tensor, int]:
    """The weight's rows; dim: their length, None: any."""
    if w.dim() != 2:
        raise ValueError(f"weight must be [units, {'dim' if dim is None else dim}], got "
                         f"{tuple(w.shape)}")
    _like(w, w.shape if dim is None else (w.shape[0], dim), x, "weight")
    return _rows(w, "weight")


def _bias(b: torch.Tensor | None, units: int, x: torch.Tensor) -> torch.Tensor | None:
    if b is None:
        return None
    _like(b, (units,), x, "bias")
    return b.contiguous()


def _aligned(t: torch.Tensor, ld: int) -> bool:
    """Whether rows start on 16-byte boundaries and are whole vectors long."""
    per = 16 // t.element_size()
    return not (t.data_ptr() % 16 or (ld | t.shape[-1]) % per)


def _workspace(tokens, dim, units, act, code, backward, aligned, device, shared):
    nbytes = library().linear_workspace_bytes(tokens, dim, units, act, code, backward, aligned)
    if nbytes == 0:
        return None, 0
    return (shared or SharedBuffer()).workspace(nbytes, device), nbytes


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               residual: torch.Tensor | None = None, kind: str | None = None,
               param: float | None = None, out: torch.Tensor | None = None,
               shared: SharedBuffer | None = None) -> torch.Tensor:
    """y = residual + f(x weight^T + bias), [..., units]; f the activation
    ``kind``, or none.  ``out`` may not be the residual.  ``shared`` lends its
    workspace."""
    act, code = _code(kind), _dtype_code(x)
    x, ldx = _rows(x, "x")
    w, ldw = _weight(weight, x, x.shape[-1])
    tokens, (units, dim) = _tokens(x), w.shape
    shape, device = (*x.shape[:-1], units), x.device
    b = _bias(bias, units, x)
    r, ldr = None, 0
    if residual is not None:
        _like(residual, shape, x, "residual")
        r, ldr = _rows(residual, "residual")
    if out is None:
        y, ldy = torch.empty(shape, dtype=x.dtype, device=device), units
    else:
        _like(out, shape, x, "out")
        y, ldy = _out_rows(out, out, "out")
        if ldy > _lib.LINEAR_MAX_LD and ldy > units:
            raise ValueError(f"the rows of out are {ldy} elements apart, more than "
                             f"{_lib.LINEAR_MAX_LD}")
    ws, nbytes = _workspace(tokens, dim, units, act, code, 0, _aligned(x, ldx) and _aligned(w, ldw),
                            device, shared)
    launch("linear_fwd", "linear_fwd", device, act, _param_value(kind, param), x.data_ptr(), ldx,
           w.data_ptr(), ldw, _ptr(b), _ptr(r), ldr, tokens, dim, units, y.data_ptr(), ldy,
           _ptr(ws), nbytes, code)
    return y


def linear_bwd(x: torch.Tensor | None, weight: torch.Tensor, dy: torch.Tensor,
               bias: torch.Tensor | None = None, kind: str | None = None,
               param: float | None = None, need_x: bool = True, need_weight: bool = True,
               need_bias: bool | None = None, shared: SharedBuffer | None = None
               ) -> tuple[torch.Tensor | None, torch.Tensor | None, torch.Tensor | None]:
    """(dx, dweight, dbias) from the input, the weight, the bias and dy = dL/dy.
    What is not needed is None; ``need_bias`` defaults to whether there is a
    bias.  (The residual's gradient is dy.)  x may be None where nothing reads it:
    no activation, and ``need_weight`` False.  ``shared`` lends its workspace."""
    if x is None and (kind is not None or need_weight):
        raise ValueError("x must be given with an activation or need_weight")
    like = dy if x is None else x
    act, code, lead = _code(kind), _dtype_code(like), like.shape[:-1]
    if x is not None:
        x, ldx = _rows(x, "x")
    w, ldw = _weight(weight, like, None if x is None else x.shape[-1])
    units, dim = w.shape
    if x is None:
        ldx = dim
    b, device = _bias(bias, units, like), like.device
    _like(dy, (*lead, units), like, "dy")
    dy, lddy = _rows(dy, "dy")
    tokens = _tokens(dy)
    if need_bias is None:
        need_bias = b is not None
    dx = torch.empty((*lead, dim), dtype=like.dtype, device=device) if need_x else None
    dw = torch.empty((units, dim), dtype=like.dtype, device=device) if need_weight else None
    db = torch.empty((units,), dtype=like.dtype, device=device) if need_bias else None
    aligned = (_lib.LINEAR_ALIGNED_XW * ((x is None or _aligned(x, ldx)) and _aligned(w, ldw))
               + _lib.LINEAR_ALIGNED_DY * _aligned(dy, lddy))
    ws, nbytes = _workspace(tokens, dim, units, act, code, 1, aligned, device, shared)
    launch("linear_bwd", "linear_bwd", device, act, _param_value(kind, param), _ptr(x), ldx,
           w.data_ptr(), ldw, _ptr(b), dy.data_ptr(), lddy, tokens, dim, units, _ptr(dx), dim,
           _ptr(dw), dim, _ptr(db), _ptr(ws), nbytes, code)
    return dx, dw, db


class LinearFn(torch.autograd.Function):
    """residual + f(x W^T + bias) keeping x, where an activation or the weight's
    gradient reads it (and references to the parameters)."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, kind, param, shared):
        reads_x = kind is not None or ctx.needs_input_grad[1]
        ctx.save_for_backward(x if reads_x else None, weight, bias)
        ctx.kind, ctx.param, ctx.shared = kind, param, shared
        return linear_fwd(x, weight, bias, residual, kind, param, shared=shared)

    @staticmethod
    @first_order
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        need = ctx.needs_input_grad  # x, weight, bias, residual, ...
        dx = dw = db = None
        if any(need[:3]):
            dx, dw, db = linear_bwd(x, weight, dy, bias, ctx.kind, ctx.param, *need[:3],
                                    shared=ctx.shared)
        return dx, dw, db, dy if need[3] else None, None, None, None


class Linear(nn.Module):
    """residual + f(x weight^T + bias) over the last dimension (dim -> units);
    ``kind`` None: no activation."""

    def __init__(self, dim: int, units: int, kind: str | None = None, param: float | None = None,
                 bias: bool = True, shared: SharedBuffer | None = None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        _code(kind)
        self.weight = nn.Parameter(torch.randn(units, dim, dtype=dtype) * dim ** -0.5)
        self.bias = nn.Parameter(torch.zeros(units, dtype=dtype)) if bias else None
        self.kind, self.param, self.shared = kind, param, shared

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        return LinearFn.apply(x, self.weight, self.bias, residual, self.kind, self.param,
                              self.shared)

    def extra_repr(self) -> str:
        units, dim = self.weight.shape
        return f"{dim}, {units}, kind={self.kind}, param={self.param}, bias={self.bias is not None}"
