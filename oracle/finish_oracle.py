"""CPU oracle for the operators that finish a transformer block -- TEST
INFRASTRUCTURE.  It shares no code with the GPU path.

The definitions in binary64 (torch on the CPU), from the inputs as the kernels
read them:

    y  = r + f(z),  z = x W^T + b
    dz = dy f'(z),  dx = dz W,  dW = dz^T x,  db = sum dz

Each function also returns, per element, the largest error a binary32
evaluation with one rounding of the result may have, in the manner of
ffn_oracle: first-order forward error analysis with u = 2^-24, sums in any
order ((k + 2) u of the sum of the terms' sizes), activations to ACT_REL, and the
result's own rounding.
"""

from __future__ import annotations

import torch

from .ffn_oracle import (ACT_REL, CURVE, SLOPE, TINY, U, act, f64, half_unit)


def _z(x, w, b):
    X, W = f64(x).flatten(0, -2), f64(w)
    k = X.shape[1]
    z, size = X @ W.t(), X.abs() @ W.abs().t()
    if b is not None:
        z, size = z + f64(b), size + f64(b).abs()
    return X, W, z, (k + 3) * U * size


def _act(z, ez, kind, p, dtype):
    """f, f' and their bounds for z known to ez."""
    if kind is None:
        return z, torch.ones_like(z), ez, torch.zeros_like(z)
    f, df = act(kind, z, p)
    rel = ACT_REL[dtype]
    scale = max(1.0, abs(p)) if kind in ("swish", "leaky_relu") else 1.0
    ef = SLOPE[kind] * scale * ez + rel * f.abs()
    # f' is a sum of terms of size up to SLOPE: its own error relative to them.
    edf = CURVE[kind] * scale * ez + rel * SLOPE[kind] * scale
    if kind in ("relu", "leaky_relu"):  # f' jumps at 0
        edf = edf + (z.abs() <= ez).to(z.dtype) * 2 * scale
    return f, df, ef, edf


def linear_forward(x, w, b, r, kind, p):
    """y [tokens, units] and its bound."""
    _, _, z, ez = _z(x, w, b)
    y, _, e, _ = _act(z, ez, kind, p, x.dtype)
    if r is not None:
        R = f64(r).reshape(y.shape)
        e = e + U * ((y + R).abs() + e)
        y = y + R
    return y, e + half_unit(y.abs() + e, x.dtype) + TINY


def linear_backward(x, w, b, dy, kind, p):
    """(dx, dW, db) and their bounds."""
    X, W, z, ez = _z(x, w, b)
    D = f64(dy).flatten(0, -2)
    dt = x.dtype
    _, df, _, edf = _act(z, ez, kind, p, dt)
    dz = D * df
    e = torch.zeros_like(dz)
    if kind is not None:
        e = D.abs() * edf + 2 * U * dz.abs()
        if dt == torch.bfloat16:
            e = e + half_unit(dz.abs() + e, dt) + TINY

    def product(a, ea, c):
        k = a.shape[1]
        v, size = a @ c, (a.abs() + ea) @ c.abs()
        bound = ea @ c.abs() + (k + 4) * U * size
        return v, bound + half_unit(v.abs() + bound, dt) + TINY

    ones = torch.ones(X.shape[0], 1, dtype=torch.float64)
    dx, ex = product(dz, e, W)
    dw, ew = product(dz.t(), e.t(), X)
    db, eb = product(dz.t(), e.t(), ones)
    return (dx, dw, db[:, 0]), (ex, ew, eb[:, 0])
