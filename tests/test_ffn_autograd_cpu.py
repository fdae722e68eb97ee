"""Autograd of the feed-forward operators' functions, with CPU formulas in the
place of the kernels (results that autograd cannot see into, as the kernels'
are)."""

import pytest
import torch

from memory_efficient_activation_amd import dense, ffn, norm
from oracle import ffn_oracle as o


def _norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None):
    with torch.no_grad():
        return tuple(t.to(x.dtype) for t in o.norm_forward(x, weight, bias, eps)[0])


def _norm_bwd(x, dy, mean, rstd, weight=None, need_params=True, out=None, shared=None,
              param_dtype=None):
    with torch.no_grad():
        dx, dw, db = (t.to(x.dtype) for t in o.norm_backward(x, dy, mean, rstd, weight)[0])
        return (dx, dw, db) if need_params else (dx, None, None)


def _unit_fwd(x, wg, wu, kind="swish", param=None, out=None, shared=None):
    with torch.no_grad():
        h = o.ffn_forward(x, wg, wu, kind, 1.0)[0]
        return h.to(x.dtype).view(*x.shape[:-1], wg.shape[0])


def _unit_bwd(x, wg, wu, dh, kind="swish", param=None, need_x=True, need_weights=True,
              need_h=False, shared=None):
    with torch.no_grad():
        dx, dwg, dwu = (t.to(x.dtype) for t in o.ffn_backward(x, wg, wu, dh, kind, 1.0)[0])
        res = (dx.view(x.shape) if need_x else None, *((dwg, dwu) if need_weights else (None, None)))
        return (*res, _unit_fwd(x, wg, wu, kind)) if need_h else res


@pytest.fixture
def formulas(monkeypatch):
    for module in (norm, ffn):
        monkeypatch.setattr(module, "layer_norm_fwd", _norm_fwd)
        monkeypatch.setattr(module, "layer_norm_bwd", _norm_bwd)
    monkeypatch.setattr(ffn, "gated_ffn_fwd", _unit_fwd)
    monkeypatch.setattr(ffn, "gated_ffn_bwd", _unit_bwd)


def modules():
    torch.manual_seed(3)
    return {"LayerNorm": norm.LayerNorm(16), "GatedUnit": ffn.GatedUnit(16, 24, "gelu"),
            "PreNormGatedFeedForward": ffn.PreNormGatedFeedForward(16, 24, "swish")}


@pytest.mark.parametrize("name", sorted(modules()))
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
    for g in graph:
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            torch.autograd.grad(g.pow(2).sum(), x, retain_graph=True)
    # In a sum with terms of its own the missing ones would go unnoticed.
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        (graph[0].pow(2).sum() + x.pow(3).sum()).backward()


def test_first_derivatives_of_the_block(formulas):
    """The stand-ins' block against the plain one (the formulas are right)."""
    m = modules()["PreNormGatedFeedForward"]
    x = torch.randn(5, 16, requires_grad=True)
    dy = torch.randn(5, 16)
    got = torch.autograd.grad(m(x), (x, *m.parameters()), dy)
    m, x, dy = m.double(), x.detach().double().requires_grad_(True), dy.double()
    wrt = (x, *m.parameters())
    n = torch.nn.functional.layer_norm(x, (16,), m.weight, m.bias, m.eps)
    plain = x + (torch.nn.functional.silu(n @ m.w_gate.t()) * (n @ m.w_up.t())) @ m.w_down.t()
    for a, b in zip(got, torch.autograd.grad(plain, wrt, dy)):
        # Binary32 sums of up to 24 products and some ten roundings on the way.
        assert float((a - b).norm()) <= 34 * 2.0 ** -24 * 10 * float(b.norm())


def test_a_block_shares_memory_only_when_asked():
    """A buffer serves one stream at a time; calls of one module from two
    streams or threads would race in one that the module made itself."""
    shared = dense.SharedBuffer()
    assert ffn.PreNormGatedFeedForward(16, 24).shared is None
    assert ffn.GatedUnit(16, 24).shared is None and norm.LayerNorm(16).shared is None
    assert ffn.PreNormGatedFeedForward(16, 24, shared=shared).shared is shared


PARTS = ("x", "weight", "bias", "w_gate", "w_up", "w_down")


@pytest.mark.parametrize("wanted", [("x",), ("w_down",), ("w_gate",), ("w_up", "w_down"), ("bias",),
                                    ("weight", "w_up"), ("x", "w_down"), PARTS], ids="-".join)
def test_the_block_computes_what_is_wanted(formulas, monkeypatch, wanted):
    """With part of it frozen the block's other gradients are the same, and
    what only frozen parts need is not computed."""
    m = modules()["PreNormGatedFeedForward"]
    x = torch.randn(5, 16)
    dy = torch.randn(5, 16)
    tensors = dict(m.named_parameters(), x=x)
    x.requires_grad_(True)
    want = dict(zip(PARTS, torch.autograd.grad(m(x), [tensors[k] for k in PARTS], dy)))
    for k in PARTS:
        tensors[k].requires_grad_(k in wanted)
    asked = []

    def unit_bwd(x, wg, wu, dh, kind, param, need_x=True, need_weights=True, need_h=False,
                 shared=None):
        asked.append((need_x, need_weights, need_h))
        return _unit_bwd(x, wg, wu, dh, kind, param, need_x, need_weights, need_h)

    def norm_bwd(x, dy, mean, rstd, weight=None, need_params=True, out=None, shared=None):
        asked.append(need_params)
        return _norm_bwd(x, dy, mean, rstd, weight, need_params)

    monkeypatch.setattr(ffn, "gated_ffn_bwd", unit_bwd)
    monkeypatch.setattr(ffn, "layer_norm_bwd", norm_bwd)
    got = torch.autograd.grad(m(x), [tensors[k] for k in wanted], dy)
    for k, g in zip(wanted, got):
        assert torch.equal(g, want[k]), k
    wanted = set(wanted)
    need_norm = bool(wanted & {"x", "weight", "bias"})
    need_unit = bool(wanted & {"w_gate", "w_up"})
    expect = [(need_norm, need_unit, "w_down" in wanted)] if need_norm or need_unit else []
    assert asked == expect + ([bool(wanted & {"weight", "bias"})] if need_norm else [])
