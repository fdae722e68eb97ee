"""More gate rows than blocks, at widths whose last chunk shares columns with a chunk
of another wave: the post norm's sums, which a block adds up over its gate rows."""

import pytest
import torch

from memory_efficient_activation_amd import residual
from test_gpu_residual import BF16, F32, check, make, present

pytestmark = pytest.mark.gpu

# (leading shape, gate rows, width, types): rows of more than 2048 values are one to a
# block, which has 512 blocks, or 256 where a row's reads are 32 KB or more; the last
# chunk's number is a multiple of 64.
CASES = [((1100,), (1100,), 2049, (BF16, BF16)), ((1100,), (1100,), 2055, (F32, BF16)),
         ((600, 3), (600,), 2561, (BF16, BF16)), ((600, 2), (600,), 4097, (BF16, BF16)),
         ((300, 4), (300,), 4097, (F32, F32)), ((300,), (300,), 7687, (F32, F32)),
         ((2, 550), (2, 550), 4103, (BF16, BF16))]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("lead,gate,n,types", CASES, ids=str)
def test_against_binary64(lead, gate, n, types, center):
    check(*make(lead, n, types, gate=gate, center=center))


@pytest.mark.parametrize("lead,gate,n,types", CASES, ids=str)
def test_repeats_bit_for_bit(lead, gate, n, types):
    x, z, dy, do, args = make(lead, n, types, gate=gate)
    y, out, stats = residual.residual_norm_fwd(x, z, **args)
    first = residual.residual_norm_bwd(y, z, dy, do, stats, **args)
    for _ in range(10):
        again = residual.residual_norm_bwd(y, z, dy, do, stats, **args)
        assert all(torch.equal(a, b) for a, b in zip(present(first), present(again)))


@pytest.mark.parametrize("lead,gate,n,types", CASES[::2], ids=str)
def test_one_parameter_of_the_post_norm(lead, gate, n, types):
    """The weight's or the bias's gradient alone, without a norm behind the border."""
    for which in (0, 1):
        x, z, dy, do, args = make(lead, n, types, norms=(True, False), gate=gate)
        args["post"] = tuple(p if i == which else None for i, p in enumerate(args["post"]))
        check(x, z, dy, do, args)
