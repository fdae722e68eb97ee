"""The product's backward at the most tokens it takes."""

import pytest
import torch

from memory_efficient_activation_amd import linear
from oracle import ffn_oracle, finish_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", [None, "sigmoid"])
def test_most_tokens(kind):
    """2^30 - 1 tokens of 8 values: dx has more tiles than one launch has blocks for."""
    torch.cuda.empty_cache()
    tokens, dim, units = (1 << 30) - 1, 8, 8
    gen = torch.Generator(device=DEV).manual_seed(6)
    dy = torch.empty(tokens, units, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    w = torch.randn(units, dim, generator=gen, device=DEV).bfloat16()
    x = None if kind is None else torch.empty(tokens, dim, dtype=torch.bfloat16,
                                              device=DEV).normal_(generator=gen)
    dx = linear.linear_bwd(x, w, dy, None, kind, need_weight=False)[0]
    torch.cuda.synchronize()
    say(f"[most tokens] {kind} done")
    some = torch.tensor([0, 1, 127, 128, 1 << 29, (1 << 29) + 1, tokens - 129, tokens - 128,
                         tokens - 2, tokens - 1], device=DEV)
    some = torch.cat([some, torch.randint(0, tokens, (5000,), generator=gen, device=DEV)])
    at = torch.zeros(len(some), dim, device=DEV).bfloat16() if x is None else x[some]
    (want, _, _), (bound, _, _) = o.linear_backward(at, w, None, dy[some], kind, 0.0)
    worst = ffn_oracle.worst(dx[some], want, bound)
    say(f"{tokens} tokens, {kind}: error over bound {worst:.3f}")
    assert worst <= 1
