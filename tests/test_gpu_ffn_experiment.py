"""The feed-forward memory experiment: what the memory-efficient chain keeps,
to the byte, and the same gradients as the plain chain."""

import pytest
import torch

from memory_efficient_activation_amd import ffn_experiment as fx

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,es,tol", [(torch.float32, 4, 1e-5),
                                          (torch.bfloat16, 2, 12 * 2.0 ** -9)])
def test_a_chain_keeps_its_inputs_and_statistics(dtype, es, tol):
    tokens, dim, hidden, blocks = 512, 256, 520, 3
    r = fx.measure(tokens, dim, hidden, blocks, dtype, reps=1)
    say(f"[ffn experiment] {r}")
    # Each block's output (the next one's input, or the result) and two
    # binary32 values a token.
    kept = blocks * tokens * (dim * es + 2 * 4)
    assert r["memory_efficient"]["retained_after_forward_bytes"] == kept
    # The plain block also keeps the normalized rows, both projections, the
    # activation and the product at the least.
    assert r["plain"]["retained_after_forward_bytes"] >= kept + blocks * tokens * (dim + 4 * hidden) * es
    # Rounding to the type some twelve times on the way through three blocks
    # and back (binary32: sums of up to 520 terms).
    assert r["memory_efficient"]["grad_rel_err_vs_f32"] <= tol
