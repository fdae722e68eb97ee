"""The binary64 oracle of layer normalization and the gated unit, pinned by
PyTorch's CPU autograd in binary64, by finite differences and by closed
forms; and planted mistakes, which the pins' comparison must see."""

import math

import pytest
import torch
import torch.nn.functional as F

from oracle import ffn_oracle as o

KINDS = {"swish": lambda t, p: t * torch.sigmoid(p * t), "relu": lambda t, p: F.relu(t),
         "leaky_relu": lambda t, p: F.leaky_relu(t, p), "sigmoid": lambda t, p: torch.sigmoid(t),
         "tanh": lambda t, p: torch.tanh(t), "gelu": lambda t, p: F.gelu(t),
         "gelu_tanh": lambda t, p: F.gelu(t, approximate="tanh")}
PARAM = {"swish": 1.3, "leaky_relu": 0.1}


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float64).float()


def test_norm_matches_autograd():
    gen = torch.Generator().manual_seed(1)
    x, dy, w, b = rnd(gen, 7, 33), rnd(gen, 7, 33), rnd(gen, 33), rnd(gen, 33)
    X, W, B = (t.double().requires_grad_(True) for t in (x, w, b))
    y = F.layer_norm(X, (33,), W, B, 1e-5)
    grads = torch.autograd.grad(y, (X, W, B), dy.double())
    (yo, mean, rstd), _ = o.norm_forward(x, w, b, 1e-5)
    assert torch.allclose(yo, y.detach(), rtol=1e-12, atol=1e-12)
    # The gradient formula for the exact statistics (passed in binary64).
    got, _ = o.norm_backward(x, dy, mean, rstd, w)
    for a, c in zip(got, grads):
        assert torch.allclose(a, c, rtol=1e-11, atol=1e-11)


def test_norm_closed_forms():
    x = torch.tensor([[1.0, 1.0, 1.0], [0.0, 3.0, 0.0]])
    (y, mean, rstd), _ = o.norm_forward(x, None, None, 0.25)
    assert torch.equal(y[0], torch.zeros(3, dtype=torch.float64))
    assert mean.tolist() == [1.0, 1.0]
    assert rstd[0] == 2.0 and abs(rstd[1] - (2.0 + 0.25) ** -0.5) < 1e-15
    # Without a weight the gradient is orthogonal to 1, and to xhat for eps 0.
    gen = torch.Generator().manual_seed(2)
    x, dy = rnd(gen, 5, 16), rnd(gen, 5, 16)
    mean, rstd = o.norm_stats(x, 0.0)
    (dx, _, _), _ = o.norm_backward(x, dy, mean, rstd, None)
    xh = (x.double() - mean[:, None]) * rstd[:, None]
    assert dx.sum(1).abs().max() < 1e-12 and (dx * xh).sum(1).abs().max() < 1e-12


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_unit_matches_autograd_and_differences(kind):
    gen = torch.Generator().manual_seed(3)
    p = PARAM.get(kind, 0.0)
    x, wg, wu, dh = rnd(gen, 5, 9), rnd(gen, 11, 9), rnd(gen, 11, 9), rnd(gen, 5, 11)
    X, G, W = (t.double().requires_grad_(True) for t in (x, wg, wu))
    h = KINDS[kind](X @ G.t(), p) * (X @ W.t())
    grads = torch.autograd.grad(h, (X, G, W), dh.double())
    ho, _ = o.ffn_forward(x, wg, wu, kind, p)
    assert torch.allclose(ho, h.detach(), rtol=1e-12, atol=1e-12)
    got, _ = o.ffn_backward(x, wg, wu, dh, kind, p)
    for a, c in zip(got, grads):
        assert torch.allclose(a, c, rtol=1e-11, atol=1e-11)
    # Central differences of <h, dh> along random directions.
    step = 2.0 ** -17
    for t, grad in ((x, got[0]), (wg, got[1]), (wu, got[2])):
        v = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        side = []
        for sgn in (1, -1):
            args = [(a.double() + sgn * step * v if a is t else a.double()) for a in (x, wg, wu)]
            f, _ = o.act(kind, args[0] @ args[1].t(), p)
            side.append((f * (args[0] @ args[2].t()) * dh.double()).sum())
        diff = float((side[0] - side[1]) / (2 * step))
        assert abs(diff - float((grad * v).sum())) < 1e-5 * max(1.0, abs(diff)), kind


def test_the_bounds_hold_for_a_binary32_evaluation_and_see_mistakes():
    gen = torch.Generator().manual_seed(4)
    x, wg, wu, dh = rnd(gen, 40, 64), rnd(gen, 24, 64), rnd(gen, 24, 64), rnd(gen, 40, 24)
    want, bound = o.ffn_backward(x, wg, wu, dh, "swish", 1.0)
    g, u = x @ wg.t(), x @ wu.t()
    s = torch.sigmoid(g)
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    good = (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x)
    for a, b, e in zip(good, want, bound):
        assert o.worst(a, b, e) < 1
    bad = [dg @ wg + du @ wg, dg @ wg, (dh * u * s) @ wg + du @ wu,
           (dh * u * s * (1 + g * s)) @ wg + du @ wu, 1.001 * good[0]]
    for a in bad:
        assert o.worst(a, want[0], bound[0]) > 1
    assert o.worst(torch.full_like(good[0], math.nan), want[0], bound[0]) == math.inf
    y, w = rnd(gen, 6, 50), rnd(gen, 50)
    (yo, mean, rstd), e = o.norm_forward(y, w, None, 1e-5)
    fine = F.layer_norm(y, (50,), w, None, 1e-5)
    assert o.worst(fine, yo, e[0]) < 1
    var1 = (y - y.mean(1, keepdim=True)) / y.std(1, keepdim=True) * w  # n - 1 in the variance
    assert o.worst(var1, yo, e[0]) > 1
    (dx, dw, db), eb = o.norm_backward(y, fine, mean.float(), rstd.float(), w)
    gg = fine * w
    xh = (y - mean.float()[:, None]) * rstd.float()[:, None]
    near = rstd.float()[:, None] * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    assert o.worst(near, dx, eb[0]) < 1
    assert o.worst(rstd.float()[:, None] * (gg - gg.mean(1, keepdim=True)), dx, eb[0]) > 1
    assert o.worst((fine * xh).sum(0), dw, eb[1]) < 1 and o.worst(gg.sum(0), db, eb[2]) > 1
