"""A border whose results get no gradient (what follows them gives none): zeros come
back, as from the other functions (the oracle's formulas in the place of the
kernels)."""

import pytest
import torch

from memory_efficient_activation_amd import residual

from test_finish_autograd_cpu import formulas  # noqa: F401  (a fixture)


class Stop(torch.autograd.Function):
    """The sum of t and other, with a gradient of other alone."""

    @staticmethod
    def forward(ctx, t, other):
        return t + other

    @staticmethod
    def backward(ctx, d):
        return None, d


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_zeros_come_back(formulas, post, pre):  # noqa: F811
    m = residual.ResidualNorm(8, post, pre, gate=0.5)
    x, z = (torch.randn(3, 8, requires_grad=True) for _ in range(2))
    other, d = torch.randn(3, 8, requires_grad=True), torch.randn(3, 8)
    out = m(x, z)
    for t in out if pre else (out,):
        got = torch.autograd.grad(Stop.apply(t, other), (other, x, z, *m.parameters()), d,
                                  retain_graph=True, allow_unused=True)
        assert torch.equal(got[0], d)
        assert all(g.shape == p.shape and g.dtype == p.dtype and not g.any()
                   for g, p in zip(got[1:], (x, z, *m.parameters())))
