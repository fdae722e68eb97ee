"""Measured cases of the transformer feed-forward operators.

Two operators, each in both directions:

* ``norm``: layer normalization over the last dimension,
  y = (x - mean) rstd weight + bias, and its gradients with the reductions
  of the weight's and the bias's gradients over the rows;
* ``ffn``: the gated feed-forward unit h = f(x Wg^T) * (x Wu^T), and its
  gradients from x, the weights and dh alone (both projections are
  recomputed, nothing of the forward is kept but x).

``own`` False computes them from elementary torch operations in binary32 and
rounds once at the end; ``own`` True calls this package.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = ("swish", "gelu", "gelu_tanh", "sigmoid", "relu")


# --------------------------------------------------------------------------
# Cases.
# --------------------------------------------------------------------------

def listed():
    def norm(name, way, rows, n, dtype, params):
        return {"name": name, "op": "norm", "way": way, "rows": rows, "n": n, "dtype": dtype,
                "params": params}

    def ffn(name, way, tokens, dim, hidden, dtype, kind):
        return {"name": name, "op": "ffn", "way": way, "tokens": tokens, "dim": dim,
                "hidden": hidden, "dtype": dtype, "kind": kind}

    return [
        # One token of generation: latency.
        norm("norm_fwd_token", "fwd", 1, 4096, "bf16", "bf16"),
        # The [8, 2048, 4096] activation of the 32-layer transformer, both
        # directions of a training step, with binary32 master parameters.
        norm("norm_fwd_transformer", "fwd", 16384, 4096, "bf16", "f32"),
        norm("norm_bwd_transformer", "bwd", 16384, 4096, "bf16", "f32"),
        # Odd width, odd number of rows: no row but the first is aligned.
        norm("norm_bwd_ragged_f32", "bwd", 4097, 1023, "f32", "f32"),
        # A channels-last feature map [64, 112, 112, 32]: many short rows.
        norm("norm_bwd_channels_last", "bwd", 802816, 32, "bf16", "bf16"),
        # One token of generation: the weights are read once, latency and
        # bandwidth.
        ffn("ffn_fwd_token", "fwd", 1, 4096, 16384, "bf16", "swish"),
        # A serving batch of single tokens, not a power of two.
        ffn("ffn_fwd_batch", "fwd", 24, 4096, 16384, "bf16", "swish"),
        # A prompt, or a step's forward, at the transformer's size.
        ffn("ffn_fwd_transformer", "fwd", 16384, 4096, 16384, "bf16", "swish"),
        # The backward of the same: the largest case.
        ffn("ffn_bwd_transformer", "bwd", 16384, 4096, 16384, "bf16", "swish"),
        # Widths that leave partial tiles and a hidden size whose rows are
        # not 16-byte aligned.
        ffn("ffn_bwd_ragged", "bwd", 777, 1000, 2730, "bf16", "gelu"),
        # Binary32 training at a small model's size.
        ffn("ffn_bwd_f32", "bwd", 2048, 1024, 4096, "f32", "gelu_tanh"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """Log-uniform; half of them multiples of 64, a quarter of 8, a quarter any."""
    v = _log(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, v // step * step)


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f32"))
    way = rng.choice(("fwd", "bwd"))
    if rng.random() < 0.4:
        n = _size(rng, 32, 16384)
        rows = _log(rng, 1, min(802816, (1 << 26) // n))
        return {"op": "norm", "way": way, "rows": rows, "n": n, "dtype": dtype,
                "params": rng.choice(("f32", dtype))}
    dim, hidden = _size(rng, 64, 4096), _size(rng, 64, 16384)
    # binary32 products cost some sixteen times bfloat16's.
    most = 16384 * 4096 * 16384 // (1 if dtype == "bf16" else 16)
    tokens = _log(rng, 1, min(16384, most // (dim * hidden)))
    return {"op": "ffn", "way": way, "tokens": tokens, "dim": dim, "hidden": hidden,
            "dtype": dtype, "kind": rng.choice(KINDS)}


# --------------------------------------------------------------------------
# Inputs.
# --------------------------------------------------------------------------

def _normal(gen, *shape, scale=1.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=gen)
    return t.mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "norm":
        rows, n, pt = case["rows"], case["n"], DTYPES[case["params"]]
        # A residual stream: channels of different size and offset, rows of
        # different size.
        scale = _normal(gen, n).abs_().add_(0.5)
        offset = _normal(gen, n, scale=0.5).add_(0.25)
        x = _normal(gen, rows, n)
        x.mul_(scale).add_(offset)
        x.mul_(torch.empty(rows, 1, device="cuda").uniform_(0.5, 2.0, generator=gen))
        state["x"] = x = x.to(dt)
        state["weight"] = _normal(gen, n, scale=0.25).add_(1.0).to(pt)
        state["bias"] = _normal(gen, n, scale=0.25).to(pt)
        if case["way"] == "bwd":
            state["dy"] = _normal(gen, rows, n).to(dt)
            # What the forward left: the statistics of the rows.
            var, mean = torch.var_mean(x.float(), dim=1, correction=0)
            state["mean"], state["rstd"] = mean, torch.rsqrt(var + EPS)
    else:
        tokens, dim, hidden = case["tokens"], case["dim"], case["hidden"]
        state["x"] = _normal(gen, tokens, dim).to(dt)
        state["wg"] = _normal(gen, hidden, dim, scale=dim ** -0.5).to(dt)
        state["wu"] = _normal(gen, hidden, dim, scale=dim ** -0.5).to(dt)
        if case["way"] == "bwd":
            state["dh"] = _normal(gen, tokens, hidden).to(dt)
    # A training or serving program lends its calls one workspace.  (Trees
    # that lack the operators still have this class.)
    from memory_efficient_activation_amd.dense import SharedBuffer
    state["shared"] = SharedBuffer()
    return state


# --------------------------------------------------------------------------
# The plain forms: elementary operations in binary32, rounded once.
# --------------------------------------------------------------------------

def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(dim=1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1) + EPS)
    y = c * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    pt = s["weight"].dtype
    return dx.to(s["x"].dtype), (dy * xhat).sum(dim=0).to(pt), dy.sum(dim=0).to(pt)


def _act(kind, g):
    """f(g) and f'(g)."""
    if kind == "swish":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    if kind == "gelu_tanh":
        k = (2.0 / math.pi) ** 0.5
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        return (0.5 * g * (1.0 + t),
                0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g))
    if kind == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s, s * (1.0 - s)
    on = (g > 0).float()
    return g * on, on


def _ffn_fwd(s):
    x = s["x"].float()
    a, _ = _act(s["case"]["kind"], x @ s["wg"].float().t())
    return (a * (x @ s["wu"].float().t())).to(s["x"].dtype)


def _ffn_bwd(s):
    x, wg, wu, dh = s["x"].float(), s["wg"].float(), s["wu"].float(), s["dh"].float()
    a, da = _act(s["case"]["kind"], x @ wg.t())
    dg = dh * (x @ wu.t()) * da
    du = dh * a
    dt = s["x"].dtype
    return (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)


def run(state):
    c = state["case"]
    if not own:
        plain = {("norm", "fwd"): _norm_fwd, ("norm", "bwd"): _norm_bwd,
                 ("ffn", "fwd"): _ffn_fwd, ("ffn", "bwd"): _ffn_bwd}
        return plain[c["op"], c["way"]](state)
    from memory_efficient_activation_amd import ffn, norm
    if c["op"] == "norm":
        if c["way"] == "fwd":
            return norm.layer_norm_fwd(state["x"], state["weight"], state["bias"], EPS)
        return norm.layer_norm_bwd(state["x"], state["dy"], state["mean"], state["rstd"],
                                   state["weight"], shared=state["shared"])
    if c["way"] == "fwd":
        return ffn.gated_ffn_fwd(state["x"], state["wg"], state["wu"], c["kind"],
                                 shared=state["shared"])
    return ffn.gated_ffn_bwd(state["x"], state["wg"], state["wu"], state["dh"], c["kind"],
                             shared=state["shared"])


# --------------------------------------------------------------------------
# What a pass cannot do without.
# --------------------------------------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        ps = 4 if case["params"] == "f32" else 2
        if case["way"] == "fwd":
            return {"bytes": 2 * rows * n * es + 2 * n * ps + 8 * rows, "flops": 8 * rows * n}
        return {"bytes": 3 * rows * n * es + 3 * n * ps + 8 * rows, "flops": 15 * rows * n}
    m, d, f = case["tokens"], case["dim"], case["hidden"]
    if case["way"] == "fwd":
        return {"bytes": (m * d + 2 * f * d + m * f) * es, "flops": 4 * m * d * f}
    return {"bytes": (2 * m * d + 4 * f * d + m * f) * es, "flops": 12 * m * d * f}


# --------------------------------------------------------------------------
# The definitions in binary64; gradients by differentiating the definition.
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        x, w, b = (s[k].to(f64).requires_grad_(case["way"] == "bwd")
                   for k in ("x", "weight", "bias"))
        if case["way"] == "fwd":
            mean = x.sum(1) / case["n"]
            rstd = ((x - mean[:, None]).square().sum(1) / case["n"] + EPS).pow(-0.5)
            return (x - mean[:, None]) * (rstd[:, None] * w) + b, mean, rstd
        # The statistics are inputs of the pass: dx has the three terms of
        # their dependence on x written as projections on 1 and on xhat.
        with torch.no_grad():
            z = (x - s["mean"].to(f64)[:, None]) * s["rstd"].to(f64)[:, None]
            dy = s["dy"].to(f64)
            q = torch.stack([(dy @ w), ((dy * z) @ w)]) / case["n"]
            dx = (dy * w - q[0][:, None] - z * q[1][:, None]) * s["rstd"].to(f64)[:, None]
            return dx, torch.einsum("rn,rn->n", dy, z), torch.ones_like(dy[:, 0]) @ dy
    funcs = {"swish": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
             "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
             "sigmoid": torch.sigmoid, "relu": torch.relu}
    x, wg, wu = (s[k].to(f64).requires_grad_(case["way"] == "bwd") for k in ("x", "wg", "wu"))
    h = funcs[case["kind"]](torch.nn.functional.linear(x, wg)) * torch.nn.functional.linear(x, wu)
    if case["way"] == "fwd":
        return h
    return torch.autograd.grad(h, (x, wg, wu), s["dh"].to(f64))
