"""Layer normalization on libmeswish (include/layer_norm.h).

y = (x - mean) rstd weight + bias over the last dimension, with
mean = sum x / n and rstd = 1 / sqrt(sum (x - mean)^2 / n + eps).  In the
manner of the memory-efficient activations the backward keeps the input and
recomputes the normalized map, from two binary32 values a row.

* ``layer_norm_fwd(x, weight, bias, eps)`` -> (y, mean, rstd);
* ``layer_norm_bwd(x, dy, mean, rstd, weight)`` -> (dx, dweight, dbias);
* ``LayerNormFn`` / ``LayerNorm`` -- an autograd function and module that
  keep x and the rows' statistics.

x is float32 or bfloat16 and may have any leading shape; rows at a constant
distance (a column range of a wider matrix) are read in place.  weight and
bias are float32 or bfloat16, independent of x.  Tensor-level functions only
check and marshal arguments; there is no CPU path.  Gradients cannot be
differentiated again (an attempt raises).
"""

from __future__ import annotations

import torch
import torch.nn as nn

from . import _lib
from ._autograd import first_order
from .dense import EPS, SharedBuffer
from .functional import _DTYPES, _dtype_code, _require_device, _same

# The current stream's handle by device index, and the current device,
# without building objects for every call (0.1 us each against 2 and 0.5 of a
# call's 10).
_raw_stream = torch._C._cuda_getCurrentRawStream
_device_index = torch._C._cuda_getDevice


def library():
    return _lib._LIB or _lib.library()


def launch(name: str, what: str, device: torch.device, *args) -> None:
    """The library's function on the device's current stream; raises on a
    status that is not zero."""
    i = device.index
    if i == _device_index():
        st = getattr(library(), name)(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            st = getattr(library(), name)(*args, _raw_stream(i))
    if st:
        _lib.check(st, what)


def as_rows(t: torch.Tensor, name: str) -> tuple[torch.Tensor, int, int, int]:
    """(t, rows, n, ld): t as rows of n contiguous elements, ld elements
    apart; copied only if its strides allow no such reading."""
    if not t.is_cuda:
        _require_device(t, name)
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    n = shape[-1]
    if t.is_contiguous():
        return t, (t.numel() // n if n else 0), n, n
    if t.stride(-1) == 1 or n == 1:
        # Every leading dimension steps over whole blocks of the next.
        ld, ok, span = None, t.numel() > 0, 1
        for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
            if size == 1:
                continue
            if ld is None:
                ld, span = stride, size
            elif stride == ld * span:
                span *= size
            else:
                ok = False
        if ok and (ld is None or ld >= n):
            return t, t.numel() // n, n, (n if ld is None else ld)
    t = t.contiguous()
    return t, (t.numel() // n if n else 0), n, n


def _param(p: torch.Tensor | None, n: int, like: torch.Tensor, name: str) -> int | None:
    if p is None:
        return None
    if p.dtype is not torch.float32 and p.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be float32 or bfloat16, got {p.dtype}")
    if p.shape != (n,) or not p.is_contiguous() or p.get_device() != like.get_device():
        raise ValueError(f"{name} must be a contiguous tensor of {n} values on {like.device}")
    return p.data_ptr()


def _out_rows(out: torch.Tensor | None, x: torch.Tensor, name: str):
    if out is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device), x.shape[-1]
    _same(x, out, "x", name)
    view, _, _, ld = as_rows(out, name)
    if view is not out:
        raise ValueError(f"{name} must have contiguous rows at a constant distance")
    return out, ld


def _param_code(weight, bias, x) -> int:
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight and bias have different dtypes ({weight.dtype}, {bias.dtype})")
    p = weight if weight is not None else bias
    return _dtype_code(x if p is None else p)


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None,
                   bias: torch.Tensor | None = None, eps: float = EPS,
                   out: torch.Tensor | None = None
                   ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, mean, rstd): y like x, mean and rstd float32, one value a row."""
    code = _dtype_code(x)
    x, rows, n, ldx = as_rows(x, "x")
    wp, bp = _param(weight, n, x, "weight"), _param(bias, n, x, "bias")
    pcode = _param_code(weight, bias, x)
    y, ldy = _out_rows(out, x, "out")
    device = x.device
    mean, rstd = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=device).unbind(0)
    launch("layer_norm_fwd", "layer_norm_fwd", device, x.data_ptr(), ldx, wp, bp, rows, n, eps,
           y.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(), code, pcode)
    return y, mean, rstd


def layer_norm_bwd(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: torch.Tensor | None = None, need_params: bool = True,
                   out: torch.Tensor | None = None, shared: SharedBuffer | None = None,
                   param_dtype: torch.dtype | None = None
                   ) -> tuple[torch.Tensor, torch.Tensor | None, torch.Tensor | None]:
    """(dx, dweight, dbias) from the input, the upstream gradient and the
    statistics the forward returned.  dweight and dbias have weight's dtype
    (without a weight ``param_dtype``, or x's if that is None); None if
    ``need_params`` is False.  ``shared`` lends its workspace."""
    code = _dtype_code(x)
    x, rows, n, ldx = as_rows(x, "x")
    dy, _, _, lddy = as_rows(dy, "dy")
    _same(x, dy, "x", "dy")
    device, lead = x.device, x.shape[:-1]
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype is not torch.float32 or t.shape != lead or t.device != device or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape "
                             f"{tuple(lead)} on {device}")
    wp = _param(weight, n, x, "weight")
    if weight is not None and param_dtype not in (None, weight.dtype):
        raise TypeError(f"weight is {weight.dtype}, param_dtype {param_dtype}")
    pdtype = weight.dtype if weight is not None else param_dtype or x.dtype
    if pdtype not in _DTYPES:
        raise TypeError(f"param_dtype must be float32 or bfloat16, got {pdtype}")
    pcode = _DTYPES[pdtype]
    dx, lddx = _out_rows(out, x, "out")
    dw = db = wsp = None
    nbytes = 0
    if need_params:
        dw, db = torch.empty((2, n), dtype=pdtype, device=device).unbind(0)
        ws = (shared or SharedBuffer()).workspace(library().layer_norm_workspace_bytes(rows, n), device)
        wsp, nbytes = ws.data_ptr(), ws.numel()
    launch("layer_norm_bwd", "layer_norm_bwd", device, x.data_ptr(), ldx, dy.data_ptr(), lddy,
           mean.data_ptr(), rstd.data_ptr(), wp, rows, n, dx.data_ptr(), lddx,
           dw.data_ptr() if need_params else None, db.data_ptr() if need_params else None, wsp,
           nbytes, code, pcode)
    return dx, dw, db


class LayerNormFn(torch.autograd.Function):
    """Layer normalization keeping x and two values a row."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, shared):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.shared = shared
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @first_order
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        need_w, need_b = ctx.needs_input_grad[1:3]
        dx, dw, db = layer_norm_bwd(x, dy, mean, rstd, weight, need_w or need_b, shared=ctx.shared,
                                    param_dtype=ctx.bias_dtype if weight is None else None)
        return dx, dw if need_w else None, db if need_b else None, None, None


class LayerNorm(nn.Module):
    """Layer normalization over the last dimension (n values), with weight
    and, unless ``bias`` is False, bias."""

    def __init__(self, n: int, eps: float = EPS, bias: bool = True,
                 shared: SharedBuffer | None = None, dtype: torch.dtype = torch.float32):
        super().__init__()
        self.weight = nn.Parameter(torch.ones(n, dtype=dtype))
        self.bias = nn.Parameter(torch.zeros(n, dtype=dtype)) if bias else None
        self.eps, self.shared = float(eps), shared

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return LayerNormFn.apply(x, self.weight, self.bias, self.eps, self.shared)

    def extra_repr(self) -> str:
        return f"{self.weight.numel()}, eps={self.eps}, bias={self.bias is not None}"
