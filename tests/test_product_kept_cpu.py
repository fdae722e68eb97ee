"""What the product's function keeps for its backward: its input where the weight's
gradient or an activation reads it (the oracle's formulas in the place of the
kernels)."""

import pytest
import torch

from memory_efficient_activation_amd import linear

from test_border_kept_cpu import N, ROWS, kept
from test_finish_autograd_cpu import formulas  # noqa: F401  (a fixture)

UNITS = 24


@pytest.mark.parametrize("kind,frozen,sizes", [(None, False, [ROWS * N]), (None, True, []),
                                               ("gelu", True, [ROWS * N])])
def test_input_of_the_product(formulas, kind, frozen, sizes):  # noqa: F811
    """x is read for the weight's gradient and under an activation."""
    torch.manual_seed(2)
    m = linear.Linear(N, UNITS, kind)
    m.weight.requires_grad_(not frozen)
    x = torch.randn(ROWS, N, requires_grad=True)
    y, got = kept(lambda: m(x), *m.parameters())
    assert got == sizes
    wrt = [x, *(p for p in m.parameters() if p.requires_grad)]
    dy = torch.randn(ROWS, UNITS)
    want = [g for g, p in zip(linear.linear_bwd(x, m.weight, dy, m.bias, kind), (x, m.weight, m.bias))
            if p.requires_grad]
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, wrt, dy), want))
