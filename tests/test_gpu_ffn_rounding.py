"""bfloat16 calls of the gated unit round h once: f and f' are evaluated on
binary32 g to 2^-14, far inside a unit of bfloat16.

2^-14: the largest of the paths' errors that act_math.h states, GELU's tail
(5e-5) with its exponent's rounding (30 units of 2^-24, thrice); the others stay
below 2e-5.  An f rounded to bfloat16 on the way would be off by up to 2^-9, and
test_ffn_rounding_oracle.py shows that this bound tells the two apart.
"""

import pytest
import torch

import memory_efficient_activation_amd as mea
from memory_efficient_activation_amd import ffn
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.mark.parametrize("kind", sorted(mea._lib.ACTS))
@pytest.mark.parametrize("tokens", [4, 40, 300])
def test_one_rounding(kind, tokens, monkeypatch):
    monkeypatch.setitem(o.ACT_REL, BF16, 2.0 ** -14)
    gen = torch.Generator().manual_seed(tokens)
    dim, hidden = 96, 264
    p = {"swish": 1.0, "leaky_relu": 0.01}.get(kind, 0.0)
    for scale in (1.0, 4.0):
        x, wg, wu, dh = (torch.randn(*s, generator=gen) * f for s, f in
                         (((tokens, dim), scale), ((hidden, dim), dim ** -0.5),
                          ((hidden, dim), dim ** -0.5), ((tokens, hidden), 1.0)))
        x, wg, wu, dh = (t.to(BF16).to(DEV) for t in (x, wg, wu, dh))
        h = ffn.gated_ffn_fwd(x, wg, wu, kind)
        dx, dwg, dwu, h2 = ffn.gated_ffn_bwd(x, wg, wu, dh, kind, need_h=True)
        want, bound = o.ffn_forward(x, wg, wu, kind, p)
        res = [o.worst(h, want, bound), o.worst(h2, want, bound)]
        want, bound = o.ffn_backward(x, wg, wu, dh, kind, p)
        res += [o.worst(g, v, e) for g, v, e in zip((dx, dwg, dwu), want, bound)]
        say(f"{tokens} {kind} x{scale}: errors over bounds " + " ".join(f"{r:.3f}" for r in res))
        assert max(res) <= 1, res
