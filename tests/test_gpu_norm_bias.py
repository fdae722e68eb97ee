"""Layer normalization with a bias and no weight: the bias's gradient in the
bias's type, whatever the input's."""

import pytest
import torch

from memory_efficient_activation_amd import norm
from oracle import ffn_oracle as o

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pdtype", [F32, BF16])
@pytest.mark.parametrize("n", [60, 512])
def test_bias_alone(dtype, pdtype, n):
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(1000, n, generator=gen).to(dtype).to(DEV).requires_grad_(True)
    b = torch.randn(n, generator=gen).to(pdtype).to(DEV).requires_grad_(True)
    dy = torch.randn(1000, n, generator=gen).to(dtype).to(DEV)
    y = norm.LayerNormFn.apply(x, None, b, 1e-5, None)
    y.backward(dy)
    assert b.grad.dtype is pdtype and x.grad.dtype is dtype
    want = o.f64(dy).sum(0)
    depth = 1000 // 512 + 160  # additions of a column: rows of a block, groups, blocks
    bound = depth * o.U * o.f64(dy).abs().sum(0)
    bound = bound + o.half_unit(want.abs() + bound, pdtype) + o.TINY
    assert o.worst(b.grad, want, bound) <= 1


def test_refusals():
    x = torch.randn(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    _, mean, rstd = norm.layer_norm_fwd(x)
    with pytest.raises(TypeError):
        norm.layer_norm_bwd(x, x, mean, rstd, param_dtype=torch.float64)
    with pytest.raises(TypeError):
        norm.layer_norm_bwd(x, x, mean, rstd, w, param_dtype=BF16)
    _, dw, db = norm.layer_norm_bwd(x.to(BF16), x.to(BF16), mean, rstd, param_dtype=F32)
    assert dw.dtype is F32 and db.dtype is F32
