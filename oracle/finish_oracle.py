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

from .ffn_oracle import ACT_REL, CURVE, SLOPE, TINY, U, act, f64, half_unit, sum_depth


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


# ---------------------------------------------------------------------------
# The border between blocks:
#
#     p = Norm(z) or z,  y = skip x + scale gate * p,  o = Norm(y)
#
#     e = dy + through(do w_pre, yhat),  dx = skip e,  t = scale e,  q = t gate
#     dz = through(q w_post, zhat) or q,  dgate = sum t p
#     dw_pre = sum do yhat, db_pre = sum do, dw_post = sum q zhat, db_post = sum q
#
#     through(c, vhat) = rstd (c - [center] mean(c) - vhat mean(c vhat))
#
# Tensors are [rows, n]; the gate [gates, n], each row for rows / gates of x.
# ---------------------------------------------------------------------------

def _vector(p, n, none):
    return torch.full((n,), none, dtype=torch.float64) if p is None else f64(p)


def _norm(v, ev, norm, center, eps):
    """Norm of v known to ev: (out, its bound, mean, bound, rstd, bound)."""
    n = v.shape[-1]
    d = sum_depth(n)
    w, b = _vector(norm[0], n, 1.0), _vector(norm[1], n, 0.0)
    mean = torch.zeros_like(v[:, :1])
    em = mean
    if center:
        mean = v.sum(-1, keepdim=True) / n
        em = (ev.sum(-1, keepdim=True) + (d + 2) * U * (v.abs() + ev).sum(-1, keepdim=True)) / n
    c = v - mean
    var = (c * c).sum(-1, keepdim=True) / n
    # A common error of all values moves no variance to first order.
    evar = ((2 * c.abs() * ev + 2 * ev * ev).sum(-1, keepdim=True) / n + 2 * em * em
            + (d + 6) * U * var)
    r = (var + eps) ** -0.5
    high = ((var - evar).clamp(min=0.0) + eps) ** -0.5 * (1 + 4 * U)
    er = high - r + 4 * U * r
    out = c * r * w + b
    e = w.abs() * ((ev + em) * high + c.abs() * er + 4 * U * c.abs() * high) \
        + 2 * U * (out.abs() + b.abs())
    return out, e, mean[:, 0], em[:, 0] + TINY, r[:, 0], er[:, 0]


def _per_row(gate, rows, n):
    if gate is None:
        return torch.ones(1, n, dtype=torch.float64)
    g = f64(gate).reshape(-1, n)
    return g.repeat_interleave(rows // g.shape[0], 0) if g.shape[0] else g


def border_forward(x, z, gate, post, pre, scale, skip, center, eps):
    """[y, o, post mean, post rstd, pre mean, pre rstd] without what is absent,
    and their bounds."""
    n = x.shape[-1]
    X, p = f64(x).reshape(-1, n), f64(z).reshape(-1, n)
    G = _per_row(gate, X.shape[0], n)
    ep = torch.zeros_like(p)
    stats = []
    if post is not None:
        p, ep, *s = _norm(p, ep, post, center, eps)
        stats += [(s[0], s[1])] * center + [(s[2], s[3])]
    sg = scale * G
    y = skip * X + sg * p
    ey = sg.abs() * (ep + 3 * U * (p.abs() + ep)) + 2 * U * (skip * X).abs() + U * y.abs()
    out = [(y, ey + half_unit(y.abs() + ey, x.dtype) + TINY)]
    if pre is not None:
        o, eo, *s = _norm(y, ey, pre, center, eps)
        out.append((o, eo + half_unit(o.abs() + eo, z.dtype) + TINY))
        stats += [(s[0], s[1])] * center + [(s[2], s[3])]
    return [v for v, _ in out + stats], [e for _, e in out + stats]


def border_backward(y, z, dy, do, stats, gate, post, pre, scale, skip, center):
    """[dx, dz, dgate, post weight's, post bias's, pre weight's, pre bias's]
    without what is absent, and their bounds.  stats: post mean, post rstd, pre
    mean, pre rstd (None where absent)."""
    n = y.shape[-1]
    Z = f64(z).reshape(-1, n)
    rows = Z.shape[0]
    d, dd = sum_depth(n), rows // 256 + 300  # rows a block adds; its groups; the blocks

    def column(s):
        return torch.zeros(rows, 1, dtype=torch.float64) if s is None else f64(s).reshape(-1, 1)

    def total(t, et, groups=1):
        """Sum over rows (each group's) of t known to et."""
        t, et = t.reshape(groups, -1, n), et.reshape(groups, -1, n)
        return t.sum(1), et.sum(1) + dd * U * (t.abs() + et).sum(1)

    def through(c, ec, h, r):
        m2 = (c * h).sum(-1, keepdim=True) / n
        e2 = (ec * h.abs() + (d + 6) * U * (c.abs() + ec) * h.abs()).sum(-1, keepdim=True) / n
        m1 = e1 = torch.zeros_like(m2)
        if center:
            m1 = c.sum(-1, keepdim=True) / n
            e1 = (ec + (d + 3) * U * (c.abs() + ec)).sum(-1, keepdim=True) / n
        v = r * (c - m1 - h * m2)
        return v, r.abs() * (ec + e1 + h.abs() * e2
                             + 8 * U * (c.abs() + ec + m1.abs() + (h * m2).abs()))

    pm, pr, nm, nr = (column(s) for s in stats)
    e = torch.zeros_like(Z) if dy is None else f64(dy).reshape(-1, n)
    ee = torch.zeros_like(e)
    of_pre = []
    if pre is not None:
        h, D, w = (f64(y).reshape(-1, n) - nm) * nr, f64(do).reshape(-1, n), _vector(pre[0], n, 1.0)
        t, et = through(D * w, U * (D * w).abs(), h, nr)
        of_pre = [(pre[0], *total(D * h, 4 * U * (D * h).abs())),
                  (pre[1], *total(D, torch.zeros_like(D)))]
        e = e + t
        ee = et + 2 * U * (e.abs() + t.abs())
    out = [(skip * e, abs(skip) * ee + U * (skip * e).abs(), y.dtype)]
    t, et = scale * e, abs(scale) * ee + U * (scale * e).abs()
    p, ep = Z, torch.zeros_like(Z)
    h = Z
    if post is not None:
        h = (Z - pm) * pr
        w, b = _vector(post[0], n, 1.0), _vector(post[1], n, 0.0)
        p = h * w + b
        ep = 4 * U * (h * w).abs() + 2 * U * (p.abs() + b.abs())
    G = _per_row(gate, rows, n)
    q, eq = t * G, et * G.abs() + U * (t * G).abs()
    of_gate = []
    if gate is not None:
        g = gate.numel() // n
        v, ev = total(t * p, et * p.abs() + (t.abs() + et) * ep + 3 * U * (t * p).abs(), g)
        of_gate = [(v.reshape(gate.shape), ev.reshape(gate.shape), gate.dtype)]
    of_post = []
    if post is not None:
        of_post = [(post[0], *total(q * h, eq * h.abs() + 4 * U * (q * h).abs())),
                   (post[1], *total(q, eq))]
        q, eq = through(q * w, eq * w.abs() + U * (q * w).abs(), h, pr)
    out.append((q, eq, z.dtype))
    out += of_gate + [(v[0], ev[0], p_.dtype) for p_, v, ev in of_post + of_pre if p_ is not None]
    return [v for v, _, _ in out], [ev + half_unit(v.abs() + ev, dt) + TINY for v, ev, dt in out]
