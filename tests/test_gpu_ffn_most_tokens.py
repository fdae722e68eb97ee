"""The gated unit at the most tokens it takes."""

import pytest
import torch

from memory_efficient_activation_amd import ffn
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_most_tokens():
    """2^30 - 1 tokens of 8 values: more tiles than one launch has blocks for."""
    torch.cuda.empty_cache()
    tokens, dim, hidden = (1 << 30) - 1, 8, 8
    gen = torch.Generator(device=DEV).manual_seed(6)
    x = torch.empty(tokens, dim, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    wg, wu = (torch.randn(hidden, dim, generator=gen, device=DEV).bfloat16() for _ in range(2))
    h = ffn.gated_ffn_fwd(x, wg, wu)
    some = torch.tensor([0, 1, 127, 128, 1 << 29, (1 << 29) + 1, tokens - 129, tokens - 128,
                         tokens - 2, tokens - 1], device=DEV)
    some = torch.cat([some, torch.randint(0, tokens, (5000,), generator=gen, device=DEV)])
    want, bound = o.ffn_forward(x[some], wg, wu, "swish", 1.0)
    worst = o.worst(h[some], want, bound)
    say(f"{tokens} tokens: error over bound {worst:.3f}")
    assert worst <= 1
