"""The activations' gradients cannot be differentiated again (CPU formulas in
the place of the kernels, which autograd does not see into either)."""

import pytest
import torch

from memory_efficient_activation_amd import module


@pytest.mark.parametrize("square", [False, True])
def test_activation_raises(monkeypatch, square):
    def fwd(kind, x, param=None):
        return torch.tanh(x).detach()

    def bwd(kind, x, dy, param=None):
        return (dy * (1 - torch.tanh(x) ** 2)).detach()

    monkeypatch.setattr(module, "act_fwd", fwd)
    monkeypatch.setattr(module, "act_bwd", bwd)
    x = torch.randn(10, requires_grad=True)

    def first(**kw):
        y = module.MemoryEfficientActivation("tanh")(x)
        return torch.autograd.grad((y * y if square else y).sum(), x, **kw)[0]

    g = first(create_graph=True)
    assert torch.equal(g, first()) and not first().requires_grad
    with pytest.raises(RuntimeError, match="ActFn.*cannot be differentiated again"):
        (g.sum() + x.sum()).backward()
