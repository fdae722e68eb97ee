"""The gated unit on rows further apart than the library takes: the last token
of each of a batch of long sequences, a weight inside a wide matrix."""

import pytest
import torch

from memory_efficient_activation_amd import _lib, ffn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_last_token_of_long_sequences(dtype):
    torch.manual_seed(0)
    x = torch.randn(3, _lib.GATED_FFN_MAX_LD // 64 + 1, 64, device=DEV).to(dtype)[:, -1]
    dh = torch.randn(3, _lib.GATED_FFN_MAX_LD // 40 + 1, 40, device=DEV).to(dtype)[:, -1]
    w = torch.randn(40, _lib.GATED_FFN_MAX_LD + 8, device=DEV).to(dtype)[:, :64]
    near = [t.contiguous() for t in (x, w, dh)]
    assert torch.equal(ffn.gated_ffn_fwd(x, w, w), ffn.gated_ffn_fwd(near[0], near[1], near[1]))
    for a, b in zip(ffn.gated_ffn_bwd(x, w, w, dh),
                    ffn.gated_ffn_bwd(near[0], near[1], near[1], near[2])):
        assert torch.equal(a, b)
    out = torch.empty(3, _lib.GATED_FFN_MAX_LD // 40 + 1, 40, device=DEV, dtype=dtype)[:, -1]
    with pytest.raises(ValueError, match="apart"):
        ffn.gated_ffn_fwd(x, w, w, out=out)


def test_block_on_the_last_token():
    torch.manual_seed(0)
    m = ffn.PreNormGatedFeedForward(64, 96, dtype=torch.bfloat16).to(DEV)
    x = torch.randn(2, 40000, 64, device=DEV, dtype=torch.bfloat16)[:, -1]
    assert torch.equal(m(x), m(x.contiguous()))
