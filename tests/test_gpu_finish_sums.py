"""Weight and bias gradients over 2^21 rows, to the row: sums of whole numbers, which
binary32 holds exactly in any order."""

import pytest
import torch

from memory_efficient_activation_amd import linear

from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
TOKENS, DIM, UNITS = (1 << 21) + 77, 1032, 1032  # past 2^31 elements


def rows(n, cols, most, dtype, seed):
    """A thousand rows of 0 .. most, repeated to n."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    few = torch.randint(0, most + 1, (1000, cols), device=DEV, generator=gen)
    return few, few.to(dtype).repeat((n + 999) // 1000, 1)[:n]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [None, "relu"])
def test_every_row_counts_once(kind, dtype):
    fx, x = rows(TOKENS, DIM, 1, dtype, 1)
    fd, dy = rows(TOKENS, UNITS, 3, dtype, 2)
    # z > 0, and relu's slope 1: no row of x is all zeros.
    w = torch.rand(UNITS, DIM, device=DEV).clamp_(min=0.25).to(dtype)
    assert bool((fx.sum(1) > 0).all())
    dw, db = linear.linear_bwd(x, w, dy, None, kind, need_x=False, need_bias=True)[1:]
    torch.cuda.synchronize()
    say(f"[sums] {kind} {dtype} done")
    times = torch.tensor([(TOKENS + 999 - i) // 1000 for i in range(1000)], dtype=torch.float64,
                         device=DEV)

    def sums(times):
        few = fd.double() * times[:, None]
        return few.t() @ fx.double(), few.sum(0)

    want = sums(times)
    # At most 3 a row: 3 (2^21 + 77) < 2^24, and every partial sum is a whole number.
    assert max(float(t.max()) for t in want) < 2.0 ** 24
    for got, t in zip((dw, db), want):
        assert torch.equal(got, t.to(dtype))  # one rounding, to nearest even
    # One row of each thousand left out, or one row in all where the result is not
    # rounded further, would be another result.
    short = times.clone()
    short[500] -= 1 if dtype is F32 else times[500]
    for t, s in zip(want, sums(short)):
        assert not torch.equal(t.to(dtype), s.to(dtype))
