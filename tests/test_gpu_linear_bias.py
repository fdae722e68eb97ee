"""The bias's gradient is the sum of dz before its rounding to the products'
operand type: as near as one rounding of the result."""

import pytest
import torch

from memory_efficient_activation_amd import dense, linear
from oracle import ffn_oracle as fo, finish_oracle as o

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
# Few tokens; a split sum; tiles of 128, some of them partial; tiles of 256.
SHAPES = [(1, 64, 96), (24, 200, 1000), (40, 2048, 72), (300, 1000, 333), (777, 264, 1000),
          (2048, 256, 4096), (3000, 72, 5000)]
PARAM = {"swish": 1.0, "leaky_relu": 0.01}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind,wide", [("gelu", 1.0), ("gelu", 6.0), ("swish", 40.0), ("tanh", 1.0),
                                       ("sigmoid", 1.0)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_error_is_one_rounding(shape, kind, wide, dtype):
    """wide: z's standard deviation; 6 and 40 meet the activations' rare branches."""
    tokens, dim, units = shape
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    x = torch.randn(tokens, dim, device=DEV, generator=gen).to(dtype)
    w = (torch.randn(units, dim, device=DEV, generator=gen) * wide * dim ** -0.5).to(dtype)
    b = torch.randn(units, device=DEV, generator=gen).to(dtype)
    dy = torch.randn(tokens, units, device=DEV, generator=gen).to(dtype)
    db = linear.linear_bwd(x, w, dy, b, kind)[2]
    only = linear.linear_bwd(x, w, dy, b, kind, need_x=False, need_weight=False)[2]
    assert torch.equal(db, only)
    X, W, D = (t.to(torch.float64) for t in (x, w, dy))
    z = X @ W.t() + b.to(torch.float64)
    p = PARAM.get(kind, 0.0)
    df = fo.act(kind, z, p)[1]
    # z's own error, f' to 2^-14 of its size (binary32: 1e-5), sums of binary32.
    ez = (dim + 3) * o.U * (X.abs() @ W.abs().t() + b.to(torch.float64).abs())
    rel = 1e-5 if dtype is F32 else 2.0 ** -14
    e = D.abs() * (o.CURVE[kind] * ez + rel * o.SLOPE[kind]) + 2 * o.U * (D * df).abs()
    want = (D * df).sum(0)
    bound = e.sum(0) + (tokens + 2) * o.U * (D * df).abs().sum(0)
    bound = (bound + o.half_unit(want.abs() + bound, dtype) + o.TINY).cpu()
    assert fo.worst(db, want.cpu(), bound) <= 1


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeats_and_lent_memory(dtype):
    """The sums have a fixed order; what the workspace held does not matter."""
    shared = dense.SharedBuffer()
    torch.manual_seed(3)
    for tokens, dim, units in SHAPES[::-1]:
        x, dy = torch.randn(tokens, dim, device=DEV).to(dtype), torch.randn(tokens, units, device=DEV).to(dtype)
        w, b = torch.randn(units, dim, device=DEV).to(dtype), torch.randn(units, device=DEV).to(dtype)
        want = linear.linear_bwd(x, w, dy, b, "gelu")
        for _ in range(2):
            got = linear.linear_bwd(x, w, dy, b, "gelu", shared=shared)
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            shared.workspace(1, torch.device(DEV)).fill_(255)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [None, "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_each_gradient_alone(shape, kind, dtype):
    """Asked for alone or in pairs, a gradient is what it is among all three: bit for
    bit in bfloat16, to the order of its sum in binary32."""
    tokens, dim, units = shape
    torch.manual_seed(tokens)
    x, w = torch.randn(tokens, dim, device=DEV).to(dtype), torch.randn(units, dim, device=DEV).to(dtype)
    b, dy = torch.randn(units, device=DEV).to(dtype), torch.randn(tokens, units, device=DEV).to(dtype)
    want = linear.linear_bwd(x, w, dy, b, kind)
    sizes = (units, tokens, tokens)  # of the sums
    for need in range(8):
        asked = [bool(need >> i & 1) for i in range(3)]
        got = linear.linear_bwd(x, w, dy, b, kind, None, *asked)
        for p, q, on, k in zip(got, want, asked, sizes):
            assert (p is None) == (not on)
            if on and dtype is BF16:
                assert torch.equal(p, q)
            elif on:
                # Two orders of a sum of k terms: the norm of the difference is at most
                # k 2^-24 of the terms', which are not larger than sqrt(k) times the sum's
                # here (random signs), twice.
                assert float((p - q).norm()) <= 2 * (k + 2) ** 1.5 * 2.0 ** -24 * float(q.norm())
