"""linear.h and residual_norm.h where offsets pass 2^31 elements: the last rows
give, bit for bit, what they give in a small call (in bfloat16)."""

import pytest
import torch

from memory_efficient_activation_amd import linear, residual
from oracle import ffn_oracle, finish_oracle as fo

from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def rows(n, cols, seed):
    """n random rows, a thousand of them repeated."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    few = torch.randn(1000, cols, device=DEV, generator=gen).to(BF16)
    return few.repeat((n + 999) // 1000, 1)[:n]


def test_product_with_many_rows():
    """2^31 elements of x and of y, and of rows that lie far apart."""
    tokens, dim, units = (1 << 21) + 77, 1032, 1032
    x, r = rows(tokens, dim, 1), rows(tokens, units, 2)
    w = torch.randn(units, dim, device=DEV).mul_(dim ** -0.5).to(BF16)
    b = torch.randn(units, device=DEV).to(BF16)
    y = linear.linear_fwd(x, w, b, r, "gelu_tanh")
    dx = linear.linear_bwd(x, w, r, b, "gelu_tanh", need_weight=False, need_bias=False)[0]
    # The same tiles in the middle of a smaller call, whose plan is the same one.
    some = 1 << 17
    first = linear.linear_fwd(x[:some], w, b, r[:some], "gelu_tanh")
    firstdx = linear.linear_bwd(x[:some], w, r[:some], b, "gelu_tanh", need_weight=False,
                                need_bias=False)[0]
    say("[large] product done")
    for got, want in ((y, first), (dx, firstdx)):
        # Row i is row i mod 1000; one whole turn, at the start and at the end.
        assert torch.equal(got[:1000], want[:1000])
        last = got[tokens - 1000:]
        at = (tokens - 1000) % 1000
        assert torch.equal(last, torch.cat([want[at:1000], want[:at]]))


def test_product_of_rows_far_apart():
    """Row distances of 2^21 elements: 2^31 elements lie between the first row
    and the last."""
    tokens, dim, units, ld = 1100, 264, 136, 1 << 21
    base = torch.empty(tokens * ld, dtype=BF16, device=DEV)
    x = base.view(tokens, ld)[:, 1:1 + dim]
    r = base.view(tokens, ld)[:, 1000:1000 + units]
    y = base.view(tokens, ld)[:, 2000:2000 + units]
    x.copy_(rows(tokens, dim, 1))
    r.copy_(rows(tokens, units, 2))
    w = torch.randn(units, dim, device=DEV).mul_(dim ** -0.5).to(BF16)
    linear.linear_fwd(x, w, None, r, "swish", out=y)
    xc, rc = x.contiguous(), r.contiguous()
    assert torch.equal(y, linear.linear_fwd(xc, w, None, rc, "swish"))
    for a, b in zip(linear.linear_bwd(x, w, r, None, "swish"), linear.linear_bwd(xc, w, rc, None, "swish")):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("n", [1024, 1031, 16000, 20000])
def test_border_with_many_rows(n):
    count = ((1 << 31) // n // 1000 + 1) * 1000
    x, z = rows(count, n, 1), rows(count, n, 2)
    gate, pw, nw = (torch.randn(n, device=DEV) for _ in range(3))
    args = gate, (pw, None), (nw, None)
    y, o, stats = residual.residual_norm_fwd(x, z, *args)
    small = residual.residual_norm_fwd(x[:1000], z[:1000], *args)
    for got, want in zip((y, o, *stats), (small[0], small[1], *small[2])):
        assert torch.equal(got[:1000], want) and torch.equal(got[-1000:], want)
    say(f"[large] border forward {count} x {n} done")
    g = residual.residual_norm_bwd(y, z, x, o, stats, *args, need_params=False)
    s = residual.residual_norm_bwd(small[0], z[:1000], x[:1000], small[1], small[2], *args,
                                   need_params=False)
    for got, want in zip(g[:2], s[:2]):
        assert torch.equal(got[:1000], want) and torch.equal(got[-1000:], want)


def test_border_of_rows_far_apart():
    rows_, n, ld = 1100, 520, 1 << 21
    base = torch.empty(rows_ * ld, dtype=BF16, device=DEV).view(rows_, ld)
    x, z = base[:, 1:1 + n], base[:, 4000:4000 + n]
    x.copy_(rows(rows_, n, 1))
    z.copy_(rows(rows_, n, 2))
    gate = torch.randn(n, device=DEV)
    got = residual.residual_norm_fwd(x, z, gate, (gate, None), (None, None))
    want = residual.residual_norm_fwd(x.contiguous(), z.contiguous(), gate, (gate, None), (None, None))
    for a, b in zip((*got[:2], *got[2]), (*want[:2], *want[2])):
        assert torch.equal(a, b)
    g = residual.residual_norm_bwd(x, z, z, x, got[2], gate, (gate, None), (None, None))
    s = residual.residual_norm_bwd(x.contiguous(), z.contiguous(), z.contiguous(), x.contiguous(),
                                   got[2], gate, (gate, None), (None, None))
    for a, b in zip(g, s):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("kind", [None, "relu"])
def test_weight_gradients_over_many_rows(kind):
    """Sums over 2^21 rows of positive values (past 2^31 elements): a row too many
    or too few of each thousand would show."""
    tokens, dim, units = (1 << 21) + 77, 1032, 1032
    x, dy = rows(tokens, dim, 1).abs_(), rows(tokens, units, 2).abs_()
    w = torch.rand(units, dim, device=DEV).to(BF16)  # z > 0: relu's slope is 1
    dw, db = linear.linear_bwd(x, w, dy, None, kind, need_x=False, need_bias=True)[1:]
    times = torch.tensor([(tokens + 999 - i) // 1000 for i in range(1000)], dtype=torch.float64, device=DEV)
    few = dy[:1000].double() * times[:, None]
    want_w, want_b = few.t() @ x[:1000].double(), few.sum(0)
    # A sum of 2^21 positive terms in any order, then a rounding to bfloat16 (half a
    # step, 2^-8): at the worst each addition is off by 2^-24 of the sum.
    for got, want in ((dw, want_w), (db, want_b)):
        off = float(((got.double() - want) / want).abs().max())
        say(f"[large] {kind}: {off:.2e}")
        assert off <= tokens * 2.0 ** -24 + 2.0 ** -8


@pytest.mark.parametrize("n", [1024, 16000])
def test_border_parameters_over_many_rows(n):
    count = ((1 << 31) // n // 1000 + 1) * 1000
    x, z = rows(count, n, 1), rows(count, n, 2)
    gate, pw, pb, nw, nb = (torch.randn(n, device=DEV) for _ in range(5))
    args = gate, (pw, pb), (nw, nb)
    y, o, stats = residual.residual_norm_fwd(x, z, *args)
    g = residual.residual_norm_bwd(y, z, x, o, stats, *args)
    some = residual.RowStats(*(s[:1000] for s in stats))
    want, bound = fo.border_backward(y[:1000], z[:1000], x[:1000], o[:1000], some, *args, 1.0, 1.0, True)
    # Every thousand rows are the same: `times` the sum.  Errors grow with it, and with
    # the number of additions on the way, rows / 256 + 300 at the most.
    times, depth = count // 1000, (count // 256 + 300) / (1000 // 256 + 300)
    for got, v, e in zip(g[2:], want[2:], bound[2:]):
        assert ffn_oracle.worst(got, v * times, e * times * depth) <= 1
