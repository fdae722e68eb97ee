"""What the border's function keeps for its backward: what it reads, and no more (the
oracle's formulas in the place of the kernels)."""

import pytest
import torch

from memory_efficient_activation_amd import residual

from test_finish_autograd_cpu import formulas  # noqa: F401  (a fixture)

ROWS, N = 6, 16


def kept(fn, *own):
    """fn's results, and the sizes of what it keeps beside the tensors `own`."""
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
        out = fn()
    return out, sorted(t.numel() for t in saved if not any(t is o for o in own))


def border(post, pre, gate, frozen=False):
    torch.manual_seed(2)
    m = residual.ResidualNorm(N, post, pre, gate=0.5 if gate else None)
    for p in m.parameters():
        p.data += 0.1 * torch.randn_like(p)
    if frozen:
        m.gate.requires_grad_(False)
    x, z = (torch.randn(ROWS, N, requires_grad=True) for _ in range(2))
    return m, x, z


# post, pre, gate (None, "learned" or "frozen"), maps kept
@pytest.mark.parametrize("post,pre,gate,maps", [
    (True, True, None, 2), (True, True, "learned", 2), (True, False, None, 1),
    (True, False, "learned", 1), (False, True, None, 1), (False, True, "frozen", 1),
    (False, True, "learned", 2)])
def test_maps_of_the_border(formulas, post, pre, gate, maps):  # noqa: F811
    m, x, z = border(post, pre, gate, gate == "frozen")
    out, sizes = kept(lambda: m(x, z), *m.parameters())
    assert sizes == [ROWS] * (2 * (post + pre)) + [ROWS * N] * maps
    # The gradients are those of the whole.
    d = [torch.randn(ROWS, N) for _ in range(1 + pre)]
    wrt = [t for t in (x, z, *m.parameters()) if t.requires_grad]
    got = torch.autograd.grad(out, wrt, d if pre else d[0])
    y, o, stats = residual.residual_norm_fwd(
        x, z, m.gate, (m.post_weight, m.post_bias) if post else None,
        (m.pre_weight, m.pre_bias) if pre else None)
    want = residual.residual_norm_bwd(
        y, z, d[0], d[1] if pre else None, stats, m.gate,
        (m.post_weight, m.post_bias) if post else None,
        (m.pre_weight, m.pre_bias) if pre else None)
    by_name = dict(zip(("x", "z", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias"), want))
    names = ["x", "z", *(k for k, p in m.named_parameters() if p.requires_grad)]
    for k, g in zip(names, got):
        assert torch.equal(g, by_name[k]), k


@pytest.mark.parametrize("use", [0, 1])
def test_one_result_without_z(formulas, use):  # noqa: F811
    """A loss that reads the stream alone, or the norm alone, where z is not kept."""
    m, x, z = border(False, True, None)
    d = torch.randn(ROWS, N)
    got = torch.autograd.grad(m(x, z)[use], (x, z), d)
    both = torch.autograd.grad(m(x, z), (x, z), [d if i == use else torch.zeros(ROWS, N)
                                                for i in range(2)])
    assert all(torch.equal(a, b) for a, b in zip(got, both))


def test_broadcast_gradient_of_what_is_not_kept(formulas):  # noqa: F811
    m, x, z = border(True, False, None)
    got = torch.autograd.grad(m(x, z).sum(), (x, z))
    want = torch.autograd.grad(m(x, z), (x, z), torch.ones(ROWS, N))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
