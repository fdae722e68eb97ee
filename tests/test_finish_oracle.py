"""The oracle of linear.h and residual_norm.h against autograd of the same
formulas and against differences, in binary64."""

import pytest
import torch

from oracle import finish_oracle as o

F64 = torch.float64
KINDS = [(None, 0.0), ("swish", 1.3), ("relu", 0.0), ("leaky_relu", 0.1), ("sigmoid", 0.0),
         ("tanh", 0.0), ("gelu", 0.0), ("gelu_tanh", 0.0)]


def plain_act(z, kind, p):
    f = torch.nn.functional
    return {None: lambda: z, "swish": lambda: z * torch.sigmoid(p * z), "relu": lambda: z.relu(),
            "leaky_relu": lambda: f.leaky_relu(z, p), "sigmoid": lambda: z.sigmoid(),
            "tanh": lambda: z.tanh(), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[kind]()


def random(gen, *shape):
    # Values of binary32, which the oracle takes.
    return torch.randn(*shape, generator=gen)


@pytest.mark.parametrize("kind,p", KINDS)
@pytest.mark.parametrize("biased", [True, False])
def test_product(kind, p, biased):
    gen = torch.Generator().manual_seed(1)
    x, w, b = random(gen, 5, 7), random(gen, 6, 7), random(gen, 6) if biased else None
    r, dy = random(gen, 5, 6), random(gen, 5, 6)
    leaves = [t.to(F64).requires_grad_(True) for t in (x, w, b) if t is not None]
    y = r.to(F64) + plain_act(leaves[0] @ leaves[1].t() + (leaves[2] if biased else 0), kind, p)
    got, bound = o.linear_forward(x, w, b, r, kind, p)
    assert float((got - y.detach()).abs().max()) <= 1e-12
    # Errors of an evaluation in binary32 are a few of its units.
    assert 0 < float(bound.max()) <= 1e-4
    want = torch.autograd.grad(y, leaves, dy.to(F64))
    grads, bounds = o.linear_backward(x, w, b, dy, kind, p)
    for g, v in zip(grads, want):
        assert float((g - v).abs().max()) <= 1e-11
    assert float((grads[2] - (want[2] if biased else grads[2])).abs().max()) <= 1e-11
    assert all(0 < float(e.max()) <= 1e-2 for e in bounds)
    # Along a direction, against differences (kinks are not crossed).
    d = random(gen, 5, 7).to(F64)
    h = 1e-6

    def loss(t):
        z = t @ w.to(F64).t() + (b.to(F64) if biased else 0)
        return float((plain_act(z, kind, p) * dy.to(F64)).sum())

    X = x.to(F64)
    diff = (loss(X + h * d) - loss(X - h * d)) / (2 * h)
    assert abs(diff - float((grads[0] * d).sum())) <= 1e-6 * max(1.0, abs(diff))


def plain_norm(v, norm, center, eps):
    w, b = norm
    c = v - v.mean(-1, keepdim=True) if center else v
    out = c / (c.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    return (out * w if w is not None else out) + (b if b is not None else 0)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("gates", [None, (), (2,), (2, 3)], ids=str)
@pytest.mark.parametrize("affine", [True, False])
def test_border(monkeypatch, post, pre, gates, affine, center):
    gen = torch.Generator().manual_seed(2)
    n, lead = 9, (2, 3)
    x, z, dy, do = (random(gen, *lead, n) for _ in range(4))
    gate = None if gates is None else random(gen, *gates, n)
    vectors = [random(gen, n) if affine else None for _ in range(4)]
    scale, skip, eps = 0.7, 1.25, 1e-3
    flat = [x, z, gate, *(v for on, v in zip((post, post, pre, pre), vectors) if on)]
    leaves = [None if t is None else t.to(F64).requires_grad_(True) for t in flat]
    it = iter(leaves)
    X, Z, G = next(it), next(it), next(it)
    of = {k: (next(it), next(it)) if on else None for k, on in (("post", post), ("pre", pre))}
    P = plain_norm(Z, of["post"], center, eps) if post else Z
    g = 1.0 if G is None else G.reshape(*G.shape[:-1], *[1] * (2 - len(gates)), n)
    Y = skip * X + scale * g * P
    outs = [Y] + ([plain_norm(Y, of["pre"], center, eps)] if pre else [])
    given = {"post": vectors[:2] if post else None, "pre": vectors[2:] if pre else None}
    got, bound = o.border_forward(x, z, gate, given["post"], given["pre"], scale, skip, center, eps)
    for a, v in zip(got, outs):
        assert float((a.reshape(v.shape) - v).abs().max()) <= 1e-12
    assert all(0 < float(e.max()) <= 1e-3 for e in bound)
    # The backward reads y and the statistics as they are stored; here in
    # binary64, whose own rounding the bounds leave out.
    half_unit = o.half_unit
    monkeypatch.setattr(o, "half_unit", lambda v, dt: half_unit(v, torch.float32))
    stats = [None] * 4
    values = iter(got[len(outs):])
    for at, on in ((0, post), (2, pre)):
        if on:
            if center:
                stats[at] = next(values)
            stats[at + 1] = next(values)
    wanted = [t for t in leaves if t is not None]
    loss = (Y * dy.to(F64)).sum() + ((outs[1] * do.to(F64)).sum() if pre else 0)
    want = torch.autograd.grad(loss, wanted)
    grads, bounds = o.border_backward(Y.detach(), z, dy, do if pre else None, stats, gate,
                                      given["post"], given["pre"], scale, skip, center)
    assert len(grads) == len(want)
    for a, v in zip(grads, want):
        assert float((a.reshape(v.shape) - v).abs().max()) <= 1e-11
    assert all(float(e.max()) <= 1e-2 for e in bounds)
