"""The ungated block's gradient of its input: the residual's share and the norm's are
added in binary32 and rounded once."""

import pytest
import torch

from memory_efficient_activation_amd import block, linear, norm
from oracle import ffn_oracle, finish_oracle as o
from test_gpu_residual import BF16, DEV, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lead,dim,hidden", [((1,), 64, 160), ((3, 67), 200, 333), ((300,), 1000, 520)],
                         ids=str)
def test_one_rounding(lead, dim, hidden, dtype):
    torch.manual_seed(4)
    m = block.PreNormFeedForward(dim, hidden, dtype=dtype).to(DEV)
    for p in m.parameters():
        p.data += 0.1 * torch.randn_like(p)
    x = (3 * torch.randn(*lead, dim, device=DEV)).to(dtype).requires_grad_(True)
    dy = torch.randn(*lead, dim, device=DEV).to(dtype)
    p = [t.detach() for t in (m.weight, m.bias, m.w1, m.b1, m.w2, m.b2)]
    # What reaches the norm, by the same calls.
    n, mean, rstd = norm.layer_norm_fwd(x.detach(), p[0], p[1], m.eps)
    da = linear.linear_bwd(None, p[4], dy, need_weight=False)[0]
    dn = linear.linear_bwd(n, p[2], da, p[3], "gelu")[0]
    grads = torch.autograd.grad(m(x), (x, m.weight, m.bias), dy)
    # The gradients of y = x and o = LN(y).
    want, bound = o.border_backward(x.detach(), x.detach(), dy, dn, (None, None, mean, rstd), None,
                                    None, (p[0], p[1]), 1.0, 1.0, True)
    for g, v, e in zip(grads, (want[0], *want[2:]), (bound[0], *bound[2:])):
        assert ffn_oracle.worst(g.flatten(0, -2) if g.dim() > 1 else g, v, e) <= 1
