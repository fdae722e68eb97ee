"""Autograd of the feed-forward modules with the kernels themselves."""

import pytest
import torch

from memory_efficient_activation_amd import ffn, norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("make", [lambda: norm.LayerNorm(16), lambda: ffn.GatedUnit(16, 24, "gelu"),
                                  lambda: ffn.PreNormGatedFeedForward(16, 24, "swish")],
                         ids=["LayerNorm", "GatedUnit", "PreNormGatedFeedForward"])
def test_second_derivatives_raise(make):
    torch.manual_seed(3)
    m = make().to(DEV)
    x = torch.randn(5, 16, device=DEV, requires_grad=True)
    wrt = (x, *m.parameters())
    for loss in (lambda y: y.sum(), lambda y: y.pow(2).sum()):
        once = torch.autograd.grad(loss(m(x)), wrt)
        graph = torch.autograd.grad(loss(m(x)), wrt, create_graph=True)
        for a, b in zip(once, graph):
            assert torch.equal(a, b)
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            (graph[0].pow(2).sum() + x.pow(3).sum()).backward()


@pytest.mark.parametrize("wanted", [("x",), ("w_down",), ("w_gate", "bias"), ("x", "w_down")],
                         ids="-".join)
def test_block_with_frozen_parts(wanted):
    torch.manual_seed(5)
    m = ffn.PreNormGatedFeedForward(72, 200, "gelu", dtype=torch.bfloat16).to(DEV)
    x = torch.randn(3, 50, 72, device=DEV).bfloat16().requires_grad_(True)
    dy = torch.randn(3, 50, 72, device=DEV).bfloat16()
    tensors = dict(m.named_parameters(), x=x)
    want = dict(zip(tensors, torch.autograd.grad(m(x), list(tensors.values()), dy)))
    for k, t in tensors.items():
        t.requires_grad_(k in wanted)
    for k, g in zip(wanted, torch.autograd.grad(m(x), [tensors[k] for k in wanted], dy)):
        assert torch.equal(g, want[k]), k
