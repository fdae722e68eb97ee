"""Autograd of the product's, the border's and the blocks' functions, with the
oracle's formulas in the place of the kernels (results that autograd cannot see
into, as the kernels' are)."""

import pytest
import torch
import torch.nn.functional as F

from memory_efficient_activation_amd import block, dense, linear, norm, residual
from oracle import finish_oracle as fo

import test_ffn_autograd_cpu as stand


def _linear_fwd(x, weight, bias=None, residual=None, kind=None, param=None, out=None, shared=None):
    with torch.no_grad():
        y = fo.linear_forward(x, weight, bias, residual, kind, 1.0)[0]
        return y.to(x.dtype).view(*x.shape[:-1], weight.shape[0])


def _linear_bwd(x, weight, dy, bias=None, kind=None, param=None, need_x=True, need_weight=True,
                need_bias=None, shared=None):
    with torch.no_grad():
        if x is None:
            assert kind is None and not need_weight
            x = dy.new_zeros(*dy.shape[:-1], weight.shape[1])
        dx, dw, db = (t.to(x.dtype) for t in
                      fo.linear_backward(x, weight, bias, dy, kind, 1.0)[0])
        need_bias = bias is not None if need_bias is None else need_bias
        return (dx.view(x.shape) if need_x else None, dw if need_weight else None,
                db if need_bias else None)


def _border_fwd(x, z, gate=None, post=None, pre=None, scale=1.0, skip=1.0, center=True, eps=1e-5):
    with torch.no_grad():
        v = [t.float() for t in fo.border_forward(x, z, gate, post, pre, scale, skip, center, eps)[0]]
        y = v.pop(0).view(x.shape)
        o = v.pop(0).view(x.shape) if pre else None
        s = [None] * 4
        for at, norm_ in ((0, post), (2, pre)):
            if norm_ is not None:
                s[at] = v.pop(0) if center else None
                s[at + 1] = v.pop(0)
        return y, o, residual.RowStats(*s)


def _border_bwd(y, z, dy, do, stats, gate=None, post=None, pre=None, scale=1.0, skip=1.0,
                center=True, need_params=True, shared=None):
    with torch.no_grad():
        v = [t.float() for t in fo.border_backward(y, z, dy, do, stats, gate, post, pre, scale,
                                                   skip, center)[0]]
        given = (gate, *(post or (None, None)), *(pre or (None, None)))
        dx, dz = v.pop(0).view(y.shape), v.pop(0).view(y.shape)
        return residual.ResidualNormGrads(
            dx, dz, *(v.pop(0) if p is not None else None for p in given)) if need_params else \
            residual.ResidualNormGrads(dx, dz, *[None] * 5)


@pytest.fixture
def formulas(monkeypatch):
    for module in (linear, block):
        monkeypatch.setattr(module, "linear_fwd", _linear_fwd)
        monkeypatch.setattr(module, "linear_bwd", _linear_bwd)
    for module in (norm, block):
        monkeypatch.setattr(module, "layer_norm_fwd", stand._norm_fwd)
        monkeypatch.setattr(module, "layer_norm_bwd", stand._norm_bwd)
    monkeypatch.setattr(block, "gated_ffn_fwd", stand._unit_fwd)
    monkeypatch.setattr(block, "gated_ffn_bwd", stand._unit_bwd)
    monkeypatch.setattr(residual, "residual_norm_fwd", _border_fwd)
    monkeypatch.setattr(residual, "residual_norm_bwd", _border_bwd)


class Border(torch.nn.Module):
    """A border as a function of one tensor, both results in one."""

    def __init__(self, n, **k):
        super().__init__()
        self.border = residual.ResidualNorm(n, **k)

    def forward(self, x):
        out = self.border(x, x.flip(0))
        return out if torch.is_tensor(out) else out[0] + 2 * out[1]


def modules():
    torch.manual_seed(3)
    return {"Linear": linear.Linear(16, 16, "gelu"), "LinearPlain": linear.Linear(16, 16, bias=False),
            "ResidualNorm": Border(16, gate=0.5), "ResidualNormPost": Border(16, pre=False),
            "PreNormFeedForward": block.PreNormFeedForward(16, 24),
            "PreNormFeedForwardNoBias": block.PreNormFeedForward(16, 24, "tanh", bias=False),
            "GatedFeedForward": block.GatedFeedForward(16, 24),
            "GatedFeedForwardStack": block.GatedFeedForwardStack(16, 24, 2, gate=0.5)}


def plain(name, m, x):
    """The modules' formulas in torch."""
    def border(e, a, z):
        p = F.layer_norm(z, (16,), e.post_weight, e.post_bias, e.eps) if e.post else z
        y = e.skip * a + e.scale * (1 if e.gate is None else e.gate) * p
        return (y, F.layer_norm(y, (16,), e.pre_weight, e.pre_bias, e.eps)) if e.pre else y

    def gated(b, n):
        return (F.silu(n @ b.w_gate.t()) * (n @ b.w_up.t())) @ b.w_down.t()

    if name.startswith("Linear"):
        z = F.linear(x, m.weight, m.bias)
        return F.gelu(z) if m.kind else z
    if name.startswith("ResidualNorm"):
        out = border(m.border, x, x.flip(0))
        return out[0] + 2 * out[1] if m.border.pre else out
    if name.startswith("PreNorm"):
        n = F.layer_norm(x, (16,), m.weight, m.bias, m.eps)
        return x + F.linear((F.gelu if m.kind == "gelu" else torch.tanh)(F.linear(n, m.w1, m.b1)),
                            m.w2, m.b2)
    if name == "GatedFeedForward":
        return gated(m, x)
    n = F.layer_norm(x, (16,), m.norm.weight, m.norm.bias, m.norm.eps)
    for b, e in zip(m.blocks, m.borders):
        x, n = border(e, x, gated(b, n))
    return n


NAMES = sorted(modules())


@pytest.mark.parametrize("name", NAMES)
def test_first_derivatives(formulas, name):
    m = modules()[name]
    for p in m.parameters():  # ones and zeros hide what is forgotten
        p.data += 0.1 * torch.randn_like(p)
    x = torch.randn(2, 5, 16, requires_grad=True)
    dy = torch.randn(2, 5, 16)
    y = m(x)
    got = torch.autograd.grad(y, (x, *m.parameters()), dy)
    m, X, dy = m.double(), x.detach().double().requires_grad_(True), dy.double()
    want_y = plain(name, m, X)
    # Up to some thirty results rounded to binary32 on the way, each of which
    # weights of a row sum of up to about 4 carry on.
    tol = 34 * 2.0 ** -24 * 16
    assert float((y - want_y).detach().norm()) <= tol * float(want_y.detach().norm())
    for a, b in zip(got, torch.autograd.grad(want_y, (X, *m.parameters()), dy)):
        assert float((a - b).norm()) <= tol * float(b.norm())


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("loss", ["linear", "square"])
def test_second_derivatives_raise(formulas, name, loss):
    m = modules()[name]
    x = torch.randn(5, 16, requires_grad=True)
    wrt = (x, *m.parameters())

    def first(**kw):
        y = m(x)
        return torch.autograd.grad(y.sum() if loss == "linear" else y.pow(2).sum(), wrt, **kw)

    once = first()
    assert not any(g.requires_grad for g in once)
    graph = first(create_graph=True)
    for a, b in zip(once, graph):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        (graph[0].pow(2).sum() + x.pow(3).sum()).backward()


@pytest.mark.parametrize("name", NAMES)
def test_frozen_parts(formulas, name):
    """Each tensor alone, and all but each: the gradients are the same."""
    m = modules()[name]
    x, dy = torch.randn(5, 16), torch.randn(5, 16)
    tensors = dict(m.named_parameters(), x=x)
    x.requires_grad_(True)
    want = dict(zip(tensors, torch.autograd.grad(m(x), list(tensors.values()), dy)))
    sets = [{k} for k in tensors] + [set(tensors) - {k} for k in tensors if len(tensors) > 1]
    for wanted in sets:
        for k, t in tensors.items():
            t.requires_grad_(k in wanted)
        names = [k for k in tensors if k in wanted]
        for k, g in zip(names, torch.autograd.grad(m(x), [tensors[k] for k in names], dy)):
            assert torch.equal(g, want[k]), (wanted, k)


def test_residual_of_the_product(formulas):
    m = linear.Linear(16, 24, "tanh")
    x, r = torch.randn(5, 16, requires_grad=True), torch.randn(5, 24, requires_grad=True)
    dy = torch.randn(5, 24)
    y = m(x, r)
    assert torch.allclose(y, r + torch.tanh(F.linear(x, m.weight, m.bias)), atol=1e-5)
    assert torch.equal(torch.autograd.grad(y, r, dy)[0], dy)


@pytest.mark.parametrize("use", ["y", "o"])
def test_one_result_of_the_border(formulas, use):
    """A loss that reads the stream alone, or the norm alone."""
    m = residual.ResidualNorm(16, gate=0.5)
    x, z = (torch.randn(5, 16, requires_grad=True) for _ in range(2))
    d = torch.randn(5, 16)
    wrt = (x, z, *m.parameters())
    k = "yo".index(use)
    got = torch.autograd.grad(m(x, z)[k], wrt, d, allow_unused=True)
    both = torch.autograd.grad(m(x, z), wrt, [d if i == k else torch.zeros(5, 16) for i in range(2)])
    for a, b in zip(got, both):
        assert torch.equal(a, b)


def test_memory_is_shared_only_when_asked():
    shared = dense.SharedBuffer()
    for make in (lambda s: linear.Linear(16, 24, shared=s), lambda s: residual.ResidualNorm(16, shared=s),
                 lambda s: block.PreNormFeedForward(16, 24, shared=s),
                 lambda s: block.GatedFeedForward(16, 24, shared=s)):
        assert make(None).shared is None and make(shared).shared is shared
    stack = block.GatedFeedForwardStack(16, 24, 2, shared=shared)
    assert all(m.shared is shared for m in (stack.norm, *stack.blocks, *stack.borders))


def test_settings_are_refused():
    with pytest.raises(ValueError):
        block.PreNormFeedForward(16, 24, "unknown")
    with pytest.raises(ValueError):
        block.GatedFeedForward(16, 24, "unknown")
    with pytest.raises(ValueError):
        linear.Linear(16, 24, "unknown")
    with pytest.raises(ValueError, match="at least one"):
        residual.ResidualNorm(16, post=False, pre=False)
    x = torch.randn(3, 4)
    with pytest.raises(ValueError, match="x must be given"):
        linear.linear_bwd(None, x, x)
    with pytest.raises(ValueError, match="x must be given"):
        linear.linear_bwd(None, x, x, kind="gelu", need_weight=False)
    with pytest.raises(RuntimeError, match="must be on a HIP"):
        linear.linear_bwd(None, x, x, need_weight=False)
