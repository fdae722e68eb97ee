"""The matrix product with its epilogue on the GPU against the binary64 oracle,
within bounds that the oracle derives from the formulas and types."""

import pytest
import torch

import memory_efficient_activation_amd as mea
from memory_efficient_activation_amd import dense, linear
from oracle import ffn_oracle, finish_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
PARAM = {"swish": 1.0, "leaky_relu": 0.01}
KINDS = [None, *sorted(mea._lib.ACTS)]


def make(tokens, dim, units, dtype, seed=0):
    """x, weight, bias, residual, dy."""
    gen = torch.Generator().manual_seed(seed + tokens * 7919 + dim * 131 + units)
    t = [torch.randn(tokens, dim, generator=gen),
         torch.randn(units, dim, generator=gen) * max(dim, 1) ** -0.5,
         torch.randn(units, generator=gen) * 0.5, torch.randn(tokens, units, generator=gen),
         torch.randn(tokens, units, generator=gen)]
    return [v.to(dtype).to(DEV) for v in t]


def check(x, w, b, r, dy, kind=None, param=None, shared=None):
    p = PARAM.get(kind, 0.0) if param is None else param
    y = linear.linear_fwd(x, w, b, r, kind, param, shared=shared)
    grads = linear.linear_bwd(x, w, dy, b, kind, param, need_bias=True, shared=shared)
    torch.cuda.synchronize()
    want, bound = o.linear_forward(x, w, b, r, kind, p)
    res = [ffn_oracle.worst(y, want, bound)]
    want, bound = o.linear_backward(x, w, b, dy, kind, p)
    res += [ffn_oracle.worst(g, v, e) for g, v, e in zip(grads, want, bound)]
    say(f"{tuple(x.shape)} -> {w.shape[0]} {x.dtype} {kind} bias {b is not None} residual "
        f"{r is not None}: errors over bounds " + " ".join(f"{v:.3f}" for v in res))
    assert max(res) <= 1, res
    return (y, *grads)


SHAPES = [(1, 1, 1), (1, 8, 8), (1, 64, 64), (1, 1024, 520), (2, 3, 5), (3, 100, 130),
          (8, 512, 64), (15, 96, 33), (16, 72, 200), (17, 72, 200), (24, 1000, 96),
          (31, 40, 512), (32, 512, 256), (33, 512, 256), (48, 264, 328), (64, 128, 96),
          (65, 136, 1000), (127, 64, 127), (128, 128, 64), (129, 72, 136), (200, 257, 131),
          (256, 256, 256), (257, 264, 520), (300, 512, 520), (513, 128, 384), (520, 1000, 264)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [None, "gelu"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, kind, dtype):
    check(*make(*shape, dtype), kind)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
def test_activations(kind, dtype):
    for tokens in (1, 9, 200):
        x, w, b, r, dy = make(tokens, 96, 136, dtype, seed=3)
        x *= 3  # arguments out to where every activation is flat
        check(x, w, b, r, dy, kind)
    if kind in PARAM:
        check(*make(40, 64, 80, dtype), kind, 0.3)
        check(*make(5, 64, 80, dtype), kind, -0.7)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [7, 20, 150])
def test_without_bias_or_residual(tokens, dtype):
    x, w, b, r, dy = make(tokens, 72, 104, dtype)
    for kind in (None, "tanh"):
        check(x, w, None, r, dy, kind)
        check(x, w, b, None, dy, kind)
        check(x, w, None, None, dy, kind)
    assert linear.linear_bwd(x, w, dy)[2] is None
    assert linear.linear_bwd(x, w, dy, b, need_bias=False)[2] is None
    full = linear.linear_bwd(x, w, dy, b, "swish")
    for i, name in enumerate(("need_x", "need_weight", "need_bias")):
        part = linear.linear_bwd(x, w, dy, b, "swish", **{name: False})
        assert part[i] is None
        for j in range(3):
            assert j == i or torch.equal(part[j], full[j])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(768, 512, 768), (1024, 1024, 2048), (777, 2730, 1000),
                                   (1500, 136, 2056), (4099, 128, 256), (2048, 72, 512)], ids=str)
def test_larger_shapes(shape, dtype):
    shared = dense.SharedBuffer()
    check(*make(*shape, dtype), "gelu", shared=shared)
    check(*make(*shape, dtype), None, shared=shared)


def test_many_tokens_few_units():
    check(*make(70000, 24, 40, BF16))
    check(*make(30000, 33, 17, F32), "swish")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [None, "sigmoid"])
@pytest.mark.parametrize("shape", [(1, 256, 192), (20, 96, 72), (300, 264, 320)], ids=str)
def test_strides_and_alignment(shape, kind, dtype):
    """Row distances and starts off every 16-byte boundary; leading
    dimensions; strided outputs whose neighbours stay as they were."""
    tokens, dim, units = shape
    x, w, b, r, dy = make(*shape, dtype)
    ref = check(x, w, b, r, dy, kind)

    def inside(t, left, right):
        big = torch.full((t.shape[0], t.shape[1] + left + right), float("nan"), device=DEV,
                         dtype=t.dtype)
        big[:, left:left + t.shape[1]] = t
        return big[:, left:left + t.shape[1]]

    odd = torch.full((units + 1,), float("nan"), device=DEV, dtype=dtype)[1:]
    odd.copy_(b)
    for left, right in ((1, 2), (8, 8), (0, 3)):
        check(inside(x, left, right), inside(w, left, right), odd, inside(r, right, left),
              inside(dy, left, right), kind)
        # Each alone.
        check(inside(x, left, right), w, b, r, dy, kind)
        check(x, w, b, r, inside(dy, left, right), kind)
    x3, r3 = x.view(tokens, 1, dim), r.view(tokens, 1, units)
    assert torch.equal(linear.linear_fwd(x3, w, b, r3, kind), ref[0].view(tokens, 1, units))
    for left, right in ((3, 4), (8, 0)):
        out = torch.full((tokens, units + left + right), 7.0, device=DEV, dtype=dtype)
        linear.linear_fwd(x, w, b, r, kind, out=out[:, left:left + units])
        assert torch.equal(out[:, left:left + units], ref[0])
        assert bool((out[:, :left] == 7).all()) and bool((out[:, left + units:] == 7).all())
    wt = w.t().contiguous().t()  # k strided: copied
    assert torch.equal(linear.linear_fwd(x, wt, b, r, kind), ref[0])
    wide = dy[:1].expand(tokens, units)  # one row for all tokens: copied
    check(x, w, b, r, wide, kind)


def test_empty_dimensions():
    for dtype in (F32, BF16):
        x, w, b, r, dy = make(0, 16, 24, dtype)
        assert linear.linear_fwd(x, w, b, r).shape == (0, 24)
        for kind in (None, "swish"):
            dx, dw, db = linear.linear_bwd(x, w, dy, b, kind)
            assert dx.shape == (0, 16) and dw.shape == (24, 16) and not dw.any() and not db.any()
        for tokens in (5, 50):
            x, w, b, r, dy = make(tokens, 0, 24, dtype)
            assert torch.equal(linear.linear_fwd(x, w, b, r), (r.float() + b.float()).to(dtype))
            check(x, w, b, r, dy, "sigmoid")
            x, w, b, r, dy = make(tokens, 16, 0, dtype)
            assert linear.linear_fwd(x, w, b, r).shape == (tokens, 0)
            dx, dw, db = linear.linear_bwd(x, w, dy, b)
            assert not dx.any() and dw.shape == (0, 16) and db.shape == (0,)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [5, 130, 300])
def test_non_finite_values_stay_in_their_rows(tokens, dtype):
    """A NaN token, residual or upstream row spoils its own row, a unit's weight
    or bias its own column; nothing leaks through the padding of tiles or from
    one row of a strided matrix into the next."""
    x, w, b, r, dy = make(tokens, 72, 136, dtype)
    last, nan = tokens - 1, float("nan")
    for kind in (None, "swish"):
        ref, rdx = linear.linear_fwd(x, w, b, r, kind), linear.linear_bwd(x, w, dy, b, kind)[0]
        for i in (0, 3):
            t = [x, w, b, r]
            t[i] = t[i].clone()
            t[i][last] = nan
            got = linear.linear_fwd(*t, kind)
            assert torch.equal(got[:last], ref[:last])
            assert bool(torch.isnan(got[last].float()).all())
        for i in (1, 2):
            t = [x, w, b, r]
            t[i] = t[i].clone()
            t[i][135] = nan
            got = linear.linear_fwd(*t, kind)
            assert torch.equal(got[:, :135], ref[:, :135])
            assert bool(torch.isnan(got[:, 135].float()).all())
        bad = dy.clone()
        bad[last] = nan
        dx = linear.linear_bwd(x, w, bad, b, kind)[0]
        assert torch.equal(dx[:last], rdx[:last]) and bool(torch.isnan(dx[last].float()).all())
        beside = torch.full((tokens, 200), nan, device=DEV, dtype=dtype)
        beside[:, 8:144] = dy
        got = linear.linear_bwd(x, w, beside[:, 8:144], b, kind)
        for g, v in zip(got, linear.linear_bwd(x, w, dy, b, kind)):
            assert torch.equal(g, v)


def test_repeats_bit_for_bit():
    for dtype in (F32, BF16):
        t = make(300, 264, 520, dtype)
        x, w, b, r, dy = t
        first = [linear.linear_fwd(x, w, b, r, "gelu"), *linear.linear_bwd(x, w, dy, b, "gelu")]
        for _ in range(3):
            again = [linear.linear_fwd(x, w, b, r, "gelu"), *linear.linear_bwd(x, w, dy, b, "gelu")]
            assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_autograd_and_module():
    """Module and function against binary64 autograd of the definition."""
    torch.manual_seed(0)
    for kind in (None, "gelu"):
        m = linear.Linear(48, 56, kind).to(DEV)
        with torch.no_grad():
            m.bias.normal_()
        x = torch.randn(3, 7, 48, device=DEV, requires_grad=True)
        r = torch.randn(3, 7, 56, device=DEV, requires_grad=True)
        dy = torch.randn(3, 7, 56, device=DEV)
        m(x, r).backward(dy)
        d = [t.detach().double().requires_grad_(True) for t in (x, r, m.weight, m.bias)]
        z = d[0] @ d[2].t() + d[3]
        (d[1] + (z if kind is None else torch.nn.functional.gelu(z))).backward(dy.double())
        for got, want in zip((x, r, m.weight, m.bias), d):
            err = (got.grad.double() - want.grad).norm() / want.grad.norm()
            assert float(err) < 2e-6, (kind, float(err))
        x.grad = None
        m.weight.requires_grad_(False)
        m.weight.grad = None
        m(x).backward(dy)
        assert m.weight.grad is None and x.grad is not None
        with pytest.raises(RuntimeError, match="differentiated again"):
            g, = torch.autograd.grad(m(x, r), x, dy, create_graph=True)
            g.sum().backward()


def test_streams():
    x, w, b, r, dy = make(200, 257, 131, BF16)
    ref = [linear.linear_fwd(x, w, b, r, "swish"), *linear.linear_bwd(x, w, dy, b, "swish")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [linear.linear_fwd(x, w, b, r, "swish"), *linear.linear_bwd(x, w, dy, b, "swish")]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(ref, got))


def test_refusals():
    x, w, b, r, dy = make(20, 72, 104, BF16)
    with pytest.raises(TypeError):
        linear.linear_fwd(x, w.float(), b, r)
    with pytest.raises(TypeError):
        linear.linear_fwd(x, w, b.float(), r)
    with pytest.raises(TypeError):
        linear.linear_fwd(x.half(), w.half())
    with pytest.raises(ValueError):
        linear.linear_fwd(x, w[:, :71], b, r)
    with pytest.raises(ValueError):
        linear.linear_fwd(x, w, b[:103], r)
    with pytest.raises(ValueError):
        linear.linear_fwd(x, w, b, r[:19])
    with pytest.raises(ValueError):
        linear.linear_bwd(x, w, dy[:, :103], b)
    with pytest.raises(ValueError):
        linear.linear_fwd(x, w, b, r, "softmax")
    with pytest.raises(mea.MeswishError):
        linear.linear_fwd(x, w, b, r, out=r)
    with pytest.raises(mea.MeswishError):
        linear.linear_fwd(x, w, b, r, "swish", float("nan"))
