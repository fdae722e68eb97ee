"""The border's function keeps what its backward reads, and its gradients are those of
the call with everything at hand."""

import itertools

import pytest
import torch

from memory_efficient_activation_amd import block, residual
from test_border_kept_cpu import kept
from test_gpu_residual import BF16, DEV, F32, make

pytestmark = pytest.mark.gpu
NAMES = ("x", "z", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, BF16)], ids=str)
@pytest.mark.parametrize("n", [5, 72, 3000, 9000])
@pytest.mark.parametrize("norms,gate,frozen,maps", [
    ((True, True), (), False, "yz"), ((True, False), (), False, "z"), ((True, False), None, False, "z"),
    ((False, True), None, False, "y"), ((False, True), (), True, "y"),
    ((False, True), (4,), False, "yz")], ids=str)
def test_gradients(norms, gate, frozen, maps, n, types):
    x, z, dy, do, args = make((4, 10), n, types, norms=norms, gate=gate)
    post, pre = norms
    qw, qb = args["post"] or (None, None)
    nw, nb = args["pre"] or (None, None)
    given = dict(zip(NAMES, (x, z, args["gate"], qw, qb, nw, nb)))
    y, o, stats = residual.residual_norm_fwd(x, z, **args)
    whole = residual.residual_norm_bwd(y, z, dy, do if pre else None, stats, **args)
    for name, t in given.items():
        if t is not None:
            t.requires_grad_(not (frozen and name == "gate"))
    out, sizes = kept(lambda: residual.ResidualNormFn.apply(
        x, z, args["gate"], qw, qb, nw, nb, post, pre, 1.0, 1.0, True, 1e-5, None),
        *(t for k, t in given.items() if t is not None and k not in "xz"))
    assert sizes == [40] * (2 * (post + pre)) + [40 * n] * len(maps)
    wrt = [(k, t) for k, t in given.items() if t is not None and t.requires_grad]
    grads = torch.autograd.grad(out, [t for _, t in wrt], (dy, do) if pre else dy)
    want = dict(zip(NAMES, whole))
    for (k, _), g in zip(wrt, grads):
        assert torch.equal(g, want[k]), k


def test_some_of_the_parameters():
    x, z, dy, do, args = make((3, 50), 300, gate=(3,))
    y, o, stats = residual.residual_norm_fwd(x, z, **args)
    whole = residual.residual_norm_bwd(y, z, dy, do, stats, **args)
    for need in itertools.product((False, True), repeat=5):
        some = residual.residual_norm_bwd(y, z, dy, do, stats, need_params=need, **args)
        for g, want, on in zip(some, whole, (True, True, *need)):
            assert torch.equal(g, want) if on else g is None
    for need in ((True,) * 4, (False,) * 6):
        with pytest.raises(ValueError, match="five"):
            residual.residual_norm_bwd(y, z, dy, do, stats, need_params=need, **args)


def test_stack_without_a_norm_of_the_branch():
    """Of a border the stream and two values a row alone, beside each block's input."""
    tokens, dim, blocks = 300, 264, 3
    m = block.GatedFeedForwardStack(dim, 520, blocks, post=False, dtype=BF16).to(DEV)
    x = torch.randn(tokens, dim, device=DEV).to(BF16).requires_grad_(True)
    m(x).sum().backward()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["requested_bytes.all.current"]
    y = m(x)
    kept_ = torch.cuda.memory_stats()["requested_bytes.all.current"] - before
    # The first norm's rows and values; then the stream, its norm, two values.
    assert kept_ == tokens * (dim * 2 + 8) + blocks * tokens * (2 * dim * 2 + 8)
    assert y.shape == x.shape
