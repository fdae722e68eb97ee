"""CPU oracle for layer normalization and the gated feed-forward unit -- TEST
INFRASTRUCTURE.  It shares no code with the GPU path.

Everything is the definition in binary64 (torch on the CPU), from the inputs
as the kernels read them:

    mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
    y  = (x - mean) rstd w + b
    dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy w
    dw = sum dy xhat,  db = sum dy

    h  = f(g) * u,  g = x Wg^T,  u = x Wu^T
    dg = dh u f'(g),  du = dh f(g)
    dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x

Each function also returns, per element, the largest error a binary32
evaluation with one rounding of the result may have (``bound``): first-order
forward error analysis with u = 2^-24, sums of `depth` binary32 additions
(each relative error u), and the result's own rounding.  The bounds follow
from the formulas and the types, before any kernel runs:

* a sum of products along k, added in any order: (k + 2) u sum |terms|;
* activations: relative error ACT_REL of f and of f', as the activations'
  own tests establish (1e-5 of the terms' size, binary32; 2^-9 bfloat16), the
  argument's error through the largest slope of f and f';
* bfloat16 calls round dg and du, and every result is rounded once: half a
  unit of the last place of its value (``half_unit``).
"""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24
DIGITS = {torch.float32: 24, torch.bfloat16: 8}  # of the significand
TINY = 2.0 ** -126  # results below the normal range may be flushed
ACT_REL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -9}
# Largest |f'| and |f''| of each activation (of Swish with slope a: f'' scales
# with a); ReLU and LeakyReLU jump at 0 and are treated there.
SLOPE = {"swish": 1.1, "gelu": 1.13, "gelu_tanh": 1.13, "sigmoid": 0.25, "tanh": 1.0, "relu": 1.0,
         "leaky_relu": 1.0}
CURVE = {"swish": 0.5, "gelu": 0.8, "gelu_tanh": 0.8, "sigmoid": 0.1, "tanh": 0.78, "relu": 0.0,
         "leaky_relu": 0.0}


def half_unit(v: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Half the distance between neighbouring values of the type at |v|
    (v = m 2^e, 1/2 <= m < 1: the neighbours are 2^(e - digits) apart)."""
    _, e = torch.frexp(v.abs())
    half = torch.ldexp(torch.ones_like(v), (e - DIGITS[dtype] - 1).to(torch.float64))
    return torch.where(v == 0, torch.zeros_like(v), half)


def f64(t: torch.Tensor) -> torch.Tensor:
    return t.detach().cpu().to(torch.float64)


# ---------------------------------------------------------------------------
# Layer normalization.
# ---------------------------------------------------------------------------

def sum_depth(n: int) -> int:
    """Additions any term of a row's sum passes through: at most 64 in a
    thread (n / 1024 in rows too long for registers) and 16 to combine."""
    return max(64, n // 1024 + 8) + 16


def norm_stats(x: torch.Tensor, eps: float):
    x = f64(x)
    n = x.shape[-1]
    mean = x.sum(-1) / n
    var = ((x - mean[..., None]) ** 2).sum(-1) / n
    return mean, (var + eps) ** -0.5


def norm_forward(x, w, b, eps):
    """(y, mean, rstd), (bounds of the three)."""
    dt = x.dtype
    X = f64(x)
    n = X.shape[-1]
    mean, rstd = norm_stats(x, eps)
    c = X - mean[..., None]
    W = torch.ones(n, dtype=torch.float64, device=X.device) if w is None else f64(w)
    B = torch.zeros(n, dtype=torch.float64, device=X.device) if b is None else f64(b)
    y = c * rstd[..., None] * W + B
    d = sum_depth(n)
    emean = (d + 2) * U * X.abs().sum(-1) / n
    # variance: centred squares, and the square of the mean's error.
    rel = 0.5 * ((d + 6) * U + emean ** 2 * rstd ** 2) + 4 * U
    erstd = rel * rstd
    # the mean's error moves every (x - mean) together.
    ey = ((emean * rstd)[..., None] + (c.abs() * rstd[..., None]) * (rel[..., None] + 4 * U)) \
        * W.abs() + 2 * U * (y.abs() + B.abs())
    return (y, mean, rstd), (ey + half_unit(y.abs() + ey, dt) + TINY, emean + TINY, erstd)


def norm_backward(x, dy, mean, rstd, w):
    """(dx, dw, db) for the statistics given, and their bounds."""
    dt = x.dtype
    pt = dt if w is None else w.dtype
    X, D = f64(x), f64(dy)
    n = X.shape[-1]
    mu, r = f64(mean)[..., None], f64(rstd)[..., None]
    W = torch.ones(n, dtype=torch.float64, device=X.device) if w is None else f64(w)
    xh = (X - mu) * r
    g = D * W
    m1 = g.sum(-1, keepdim=True) / n
    m2 = (g * xh).sum(-1, keepdim=True) / n
    dx = r * (g - m1 - xh * m2)
    d = sum_depth(n)
    e1 = (d + 3) * U * g.abs().sum(-1, keepdim=True) / n
    e2 = (d + 6) * U * (g * xh).abs().sum(-1, keepdim=True) / n
    edx = r.abs() * (6 * U * (g.abs() + m1.abs() + (xh * m2).abs()) + e1 + xh.abs() * e2)
    rows = X.reshape(-1, n).shape[0]
    dd = rows // 512 + 160  # rows a block adds, groups of a block, blocks
    t = (D * xh).reshape(-1, n)
    dw, db = t.sum(0), D.reshape(-1, n).sum(0)
    edw = (dd + 4) * U * t.abs().sum(0)
    edb = dd * U * D.abs().reshape(-1, n).sum(0)
    return (dx, dw, db), (edx + half_unit(dx.abs() + edx, dt) + TINY,
                          edw + half_unit(dw.abs() + edw, pt) + TINY,
                          edb + half_unit(db.abs() + edb, pt) + TINY)


# ---------------------------------------------------------------------------
# The gated unit.
# ---------------------------------------------------------------------------

def act(kind: str, g: torch.Tensor, p: float):
    """f(g) and f'(g) in binary64."""
    if kind == "swish":
        s = torch.sigmoid(p * g)
        return g * s, s * (1 + p * g * (1 - s))
    if kind == "relu":
        return torch.where(g > 0, g, 0 * g), (g > 0).to(g.dtype)
    if kind == "leaky_relu":
        return torch.where(g > 0, g, p * g), torch.where(g > 0, torch.ones_like(g),
                                                         torch.full_like(g, p))
    if kind == "sigmoid":
        s = torch.sigmoid(g)
        return s, s * torch.sigmoid(-g)
    if kind == "tanh":
        t = torch.tanh(g)
        return t, 1 / torch.cosh(g) ** 2
    if kind == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        u = k * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(2 * u)
        return g * s, s * (1 + g * (1 - s) * 2 * k * (1 + 3 * 0.044715 * g * g))
    raise ValueError(kind)


def _projections(x, wg, wu, kind, p):
    X, G, W = f64(x), f64(wg), f64(wu)
    X = X.reshape(-1, X.shape[-1])
    k = X.shape[1]
    g, u = X @ G.t(), X @ W.t()
    eg = (k + 2) * U * (X.abs() @ G.abs().t())
    eu = (k + 2) * U * (X.abs() @ W.abs().t())
    f, df = act(kind, g, p)
    rel = ACT_REL[x.dtype]
    scale = max(1.0, abs(p)) if kind in ("swish", "leaky_relu") else 1.0
    ef = SLOPE[kind] * scale * eg + rel * f.abs()
    # f' is a sum of terms of size up to SLOPE: its own error relative to them.
    edf = CURVE[kind] * scale * eg + rel * SLOPE[kind] * scale
    if kind in ("relu", "leaky_relu"):
        edf = edf + (g.abs() <= eg).to(g.dtype) * 2 * scale
    return X, G, W, g, u, f, df, eg, eu, ef, edf


def ffn_forward(x, wg, wu, kind, p):
    """h [tokens, hidden] and its bound."""
    _, _, _, _, u, f, _, _, eu, ef, _ = _projections(x, wg, wu, kind, p)
    h = f * u
    e = ef * (u.abs() + eu) + f.abs() * eu
    return h, e + half_unit(h.abs() + e, x.dtype) + TINY


def ffn_backward(x, wg, wu, dh, kind, p):
    """(dx, dWg, dWu) and their bounds."""
    X, G, W, _, u, f, df, _, eu, ef, edf = _projections(x, wg, wu, kind, p)
    D = f64(dh).reshape(-1, G.shape[0])
    dt = x.dtype
    dg, du = D * u * df, D * f
    edg = D.abs() * (eu * (df.abs() + edf) + u.abs() * edf) + 3 * U * dg.abs()
    edu = D.abs() * ef + 2 * U * du.abs()
    if dt == torch.bfloat16:
        edg = edg + half_unit(dg.abs() + edg, dt) + TINY
        edu = edu + half_unit(du.abs() + edu, dt) + TINY

    def product(a, ea, b, k):
        e = ea @ b.abs() + (k + 4) * U * (a.abs() @ b.abs())
        return a @ b, e

    k = 2 * G.shape[0]
    d1, e1 = product(dg, edg, G, k)
    d2, e2 = product(du, edu, W, k)
    dwg, ewg = product(dg.t(), edg.t(), X, X.shape[0])
    dwu, ewu = product(du.t(), edu.t(), X, X.shape[0])
    out = []
    for v, e in ((d1 + d2, e1 + e2), (dwg, ewg), (dwu, ewu)):
        out.append((v, e + half_unit(v.abs() + e, dt) + TINY))
    return tuple(v for v, _ in out), tuple(e for _, e in out)


def worst(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor) -> float:
    """Largest error over its bound; infinity where one is NaN alone."""
    got = f64(got).reshape(want.shape)
    if got.numel() == 0:
        return 0.0
    if not torch.equal(torch.isnan(got), torch.isnan(want)):
        return math.inf
    ratio = (got - want).abs() / bound
    ratio = torch.where(torch.isnan(want) | (got == want), torch.zeros_like(ratio), ratio)
    return float(ratio.max())
