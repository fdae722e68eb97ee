"""The bound that test_gpu_ffn_rounding.py sets on h tells one rounding from two
(planted in the oracle's own values)."""

import pytest
import torch

from oracle import ffn_oracle as o

BF16 = torch.bfloat16


@pytest.mark.parametrize("kind", ["swish", "gelu", "gelu_tanh", "sigmoid", "tanh"])
def test_an_activation_rounded_to_bf16_is_seen(kind, monkeypatch):
    monkeypatch.setitem(o.ACT_REL, BF16, 2.0 ** -14)
    gen = torch.Generator().manual_seed(1)
    x, wg, wu = ((torch.randn(*s, generator=gen) * f).to(BF16) for s, f in
                 (((40, 96), 1.0), ((264, 96), 96 ** -0.5), ((264, 96), 96 ** -0.5)))
    want, bound = o.ffn_forward(x, wg, wu, kind, 1.0)
    g, u = o.f64(x) @ o.f64(wg).t(), o.f64(x) @ o.f64(wu).t()
    f = o.act(kind, g, 1.0)[0]
    assert o.worst((f * u).to(BF16), want, bound) <= 1
    assert o.worst((f.to(BF16).double() * u).to(BF16), want, bound) > 1
    assert o.worst((f * u.to(BF16).double()).to(BF16), want, bound) > 1
