"""Layer normalization's backward where mean times rstd leaves binary32 though
every normalized value is finite: only the formulas' own NaN may come out.

The statistics are inputs of the backward.  A constant row of c has mean c and
any large rstd its eps gives, and xhat is zero; a row that differs from its mean
by a few units in the last place has xhat of order one.  Widths leave threads
of a group without columns, and columns that end inside a vector.
"""

import pytest
import torch

from memory_efficient_activation_amd import norm
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
WIDTHS = [1, 2, 3, 5, 7, 8, 9, 15, 17, 30, 33, 63, 65, 100, 250, 257, 500, 515, 1000, 1030, 2050,
          3000, 4100, 8000, 9000, 16380, 17000]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("params", [False, True])
def test_large_means(dtype, params):
    for n in WIDTHS:
        gen = torch.Generator().manual_seed(n)
        rows = 7
        c = 2.0 ** 121
        mean, rstd = torch.full((rows,), c), torch.full((rows,), 316.0)
        x = torch.full((rows, n), c)
        # Rows 1, 3, 5: c (1 + k 2^-7), k small (exact in both types), and
        # rstd the inverse of that step: xhat is k.
        k = torch.randint(-3, 4, (rows, n), generator=gen).float()
        mean[1::2], rstd[1::2] = c, 2.0 ** -114
        x[1::2] = c * (1 + k[1::2] * 2.0 ** -7)
        # Row 5 smaller, with a larger rstd: the same product of the two.
        x[5], mean[5], rstd[5] = 2.0 ** 100, 2.0 ** 100, 2.0 ** 60
        dy = torch.randn(rows, n, generator=gen)
        w = (1 + 0.25 * torch.randn(n, generator=gen)).to(DEV) if params else None
        x, dy, mean, rstd = x.to(dtype).to(DEV), dy.to(dtype).to(DEV), mean.to(DEV), rstd.to(DEV)
        got = norm.layer_norm_bwd(x, dy, mean, rstd, w)
        want, bound = o.norm_backward(x, dy, mean, rstd, w)
        res = [o.worst(g, v, e) for g, v, e in zip(got, want, bound)]
        say(f"width {n} {dtype}: errors over bounds {res}")
        assert max(res) <= 1, (n, res)
