"""Layer normalization at the ends of the documented sizes: rows of so many
elements, and so many long rows, that one launch cannot have threads for all
(2^32 of them).

With one row, dbias is dy and dweight is dy xhat, element by element, so every
index of the reductions shows; guards behind the outputs stay as they were.
"""

import pytest
import torch

from memory_efficient_activation_amd import norm
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
SLICE = 1 << 26
GUARD = 64


def guarded(n, dtype):
    """A row of n with values behind it that no kernel may write."""
    t = torch.empty(n + GUARD, dtype=dtype, device=DEV)
    t[n:] = 7.0
    return t


def one_row(n, dtype):
    torch.cuda.empty_cache()
    gen = torch.Generator(device=DEV).manual_seed(21)
    xs, ys, dxs = (guarded(n, dtype) for _ in range(3))
    x, y, dx = (t[:n].view(1, n) for t in (xs, ys, dxs))
    x.normal_(generator=gen).add_(0.25)
    dy = torch.empty(1, n, dtype=dtype, device=DEV).normal_(generator=gen)
    w = torch.empty(n, dtype=dtype, device=DEV).uniform_(0.5, 1.5, generator=gen)
    say(f"one row of {n} {dtype}: forward")
    _, mean, rstd = norm.layer_norm_fwd(x, w, None, out=y)
    torch.cuda.synchronize()
    say("backward")
    _, dw, db = norm.layer_norm_bwd(x, dy, mean, rstd, w, out=dx)
    torch.cuda.synchronize()
    for t in (xs, ys, dxs):
        assert bool((t[n:] == 7).all())
    assert torch.equal(db, dy[0])  # one addition to zero, and no rounding
    # Sums of the row, in binary64 a slice at a time.
    parts = range(0, n, SLICE)
    m = mean.double()
    r = rstd.double()
    sums = torch.zeros(7, dtype=torch.float64, device=DEV)
    for i in parts:
        v, d, k = x[0, i:i + SLICE].double(), dy[0, i:i + SLICE].double(), w[i:i + SLICE].double()
        g, xh = d * k, (v - m) * r
        sums += torch.stack([v.sum(), v.abs().sum(), ((v - 0.25) ** 2).sum(), g.sum(),
                             (g * xh).sum(), g.abs().sum(), (g * xh).abs().sum()])
    mu = sums[0] / n
    var = sums[2] / n - (mu - 0.25) ** 2
    depth = o.sum_depth(n)
    emean = (depth + 2) * o.U * sums[1] / n
    assert float((m[0] - mu).abs()) <= float(emean)
    rel = 0.5 * ((depth + 6) * o.U + float(emean) ** 2 / float(var)) + 4 * o.U
    assert abs(float(r[0]) * float(var + 1e-5) ** 0.5 - 1) <= rel
    # The outputs, from the statistics the forward returned.
    m1, m2 = sums[3] / n, sums[4] / n
    e1 = (depth + 3) * o.U * sums[5] / n
    e2 = (depth + 6) * o.U * sums[6] / n
    worst = [0.0, 0.0, 0.0]
    for i in parts:
        v, d, k = x[0, i:i + SLICE].double(), dy[0, i:i + SLICE].double(), w[i:i + SLICE].double()
        g, xh = d * k, (v - m) * r
        wants = (xh * k, 5 * o.U * ((v.abs() + m.abs()) * r * k)), \
            (r * (g - m1 - xh * m2),
             r * (6 * o.U * (g.abs() + m1.abs() + (xh * m2).abs()) + e1 + xh.abs() * e2)), \
            (d * xh, 4 * o.U * (d * (v.abs() + m.abs()) * r).abs())
        for j, ((want, e), got) in enumerate(zip(wants, (y[0], dx[0], dw))):
            e = e + torch.ldexp(torch.ones_like(want),
                                torch.frexp(want.abs() + e)[1] - o.DIGITS[dtype] - 1) + o.TINY
            worst[j] = max(worst[j], float(((got[i:i + SLICE].double() - want).abs() / e).max()))
    say(f"errors over bounds of y, dx, dweight: {worst}")
    assert max(worst) <= 1


@pytest.mark.parametrize("n,dtype", [((1 << 26) + 1, BF16), ((1 << 26) + 1, F32)], ids=str)
def test_more_columns_than_one_launch_reduces(n, dtype):
    one_row(n, dtype)


@pytest.mark.parametrize("n,dtype", [(16385, BF16), (8193, F32)], ids=str)
def test_more_long_rows_than_blocks(n, dtype):
    """2^22 rows and some of the kernels with a block of 1024 threads a row, in
    place (x, y, dy and dx share one matrix of 137 GB)."""
    torch.cuda.empty_cache()
    rows = (1 << 22) + 3
    gen = torch.Generator(device=DEV).manual_seed(22)
    x = torch.empty(rows, n, dtype=dtype, device=DEV)
    some = [0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 1, 1 << 22, rows - 1]
    x.fill_(1.0)  # the rows that are not looked at
    for i in some:
        x[i].normal_(generator=gen)
    keep = x[some].clone()
    say(f"{rows} rows of {n} {dtype}: forward")
    _, mean, rstd = norm.layer_norm_fwd(x, None, None, out=x)
    torch.cuda.synchronize()
    want, bound = o.norm_forward(keep, None, None, 1e-5)
    res = [o.worst(g[some], v, e) for g, v, e in zip((x, mean, rstd), want, bound)]
    y = x[some].clone()
    say("backward")
    norm.layer_norm_bwd(x, x, mean, rstd, need_params=False, out=x)
    torch.cuda.synchronize()
    want, bound = o.norm_backward(y, y, mean[some], rstd[some], None)
    res.append(o.worst(x[some], want[0], bound[0]))
    say(f"errors over bounds {res}")
    assert max(res) <= 1


@pytest.mark.parametrize("n,dtype", [((1 << 30) + 5, F32), ((1 << 31) - 8, BF16),
                                     ((1 << 31) - 1, BF16)], ids=str)
def test_columns_whose_indexes_pass_31_bits(n, dtype):
    """Past 2^30 twice a column's index (dbias's partial sums lie behind
    dweight's), and within a vector of 2^31, the longest row, a column's index
    plus the vector's length."""
    one_row(n, dtype)
