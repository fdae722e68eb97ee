"""Layer normalization on the GPU against the binary64 oracle, within bounds
that the oracle derives from the formulas and types."""

import pytest
import torch

import memory_efficient_activation_amd as mea
from memory_efficient_activation_amd import dense, norm
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def make(rows, n, dtype, pdtype, seed=0):
    gen = torch.Generator().manual_seed(seed + rows * 131 + n)
    x = torch.randn(rows, n, generator=gen) * (1 + torch.rand(rows, 1, generator=gen)) + 0.5
    dy = torch.randn(rows, n, generator=gen)
    w = 1 + 0.25 * torch.randn(n, generator=gen)
    b = 0.25 * torch.randn(n, generator=gen)
    return x.to(dtype).to(DEV), dy.to(dtype).to(DEV), w.to(pdtype).to(DEV), b.to(pdtype).to(DEV)


def check(x, dy, w, b, eps=1e-5, shared=None):
    y, mean, rstd = norm.layer_norm_fwd(x, w, b, eps)
    dx, dw, db = norm.layer_norm_bwd(x, dy, mean, rstd, w, shared=shared)
    torch.cuda.synchronize()
    want, bound = o.norm_forward(x, w, b, eps)
    res = [o.worst(g, v, e) for g, v, e in zip((y, mean, rstd), want, bound)]
    want, bound = o.norm_backward(x, dy, mean, rstd, w)
    res += [o.worst(g, v, e) for g, v, e in zip((dx, dw, db), want, bound)]
    assert y.dtype == x.dtype and dx.dtype == x.dtype
    say(f"{tuple(x.shape)} {x.dtype} {None if w is None else w.dtype}: errors over bounds "
        + " ".join(f"{r:.3f}" for r in res))
    assert max(res) <= 1, res
    return y, mean, rstd, dx, dw, db


# Rows on both sides of every choice of threads per row, in both types.
WIDTHS = [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 128, 255, 256, 257, 511, 512, 513, 1023, 1024,
          1025, 2048, 2056, 4096, 4100, 8192, 8200, 16384, 16392, 32768, 33000]


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
def test_widths(dtype, pdtype):
    for n in WIDTHS:
        for rows in (1, 5, 70) if n <= 4100 else (3,):
            check(*make(rows, n, dtype, pdtype))


@pytest.mark.parametrize("rows", [2, 255, 513, 4097, 70001])
@pytest.mark.parametrize("n,dtype", [(24, BF16), (32, BF16), (96, F32), (300, BF16), (1023, F32)])
def test_many_rows(rows, n, dtype):
    """Every block of the backward gets several batches and a partial one."""
    if rows * n > 5_000_000:
        rows = 5_000_000 // n
    check(*make(rows, n, dtype, F32), shared=dense.SharedBuffer())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_beyond_the_registers(dtype):
    check(*make(600, 40001, dtype, F32))
    check(*make(2, 300000, dtype, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [30, 520, 4096])
def test_strides_and_alignment(dtype, n):
    """Column ranges of a wider matrix, off every 16-byte boundary, and
    leading dimensions that do and do not collapse."""
    rows = 12
    wide = torch.randn(rows, n + 11, device=DEV).to(dtype)
    wdy = torch.randn(rows, n + 5, device=DEV).to(dtype)
    _, _, w, b = make(1, n + 1, dtype, F32)
    w, b = w[1:], b[1:]  # off a 16-byte boundary too
    x, dy = wide[:, 3:3 + n], wdy[:, 1:1 + n]
    assert norm.as_rows(x, "x")[0] is x
    got = check(x, dy, w, b)
    ref = check(x.contiguous(), dy.contiguous(), w.clone(), b.clone())
    for a, c in zip(got, ref):
        assert torch.equal(a, c)
    y3 = norm.layer_norm_fwd(wide.view(3, 4, n + 11)[..., 3:3 + n], w, b)[0]
    assert torch.equal(y3.view(rows, n), ref[0])
    t = torch.randn(4, n, 3, device=DEV).to(dtype).transpose(1, 2)  # copied
    yt = norm.layer_norm_fwd(t, w, b)[0]
    assert torch.equal(yt, norm.layer_norm_fwd(t.contiguous(), w, b)[0])
    one = x[:1].expand(rows, n)  # rows at distance zero
    assert torch.equal(norm.layer_norm_fwd(one, w, b)[0], ref[0][:1].expand(rows, n))
    # A strided output, neighbours untouched; and in place.
    out = torch.full((rows, n + 11), 7.0, device=DEV, dtype=dtype)
    norm.layer_norm_fwd(x, w, b, out=out[:, 5:5 + n])
    assert torch.equal(out[:, 5:5 + n], ref[0])
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 5 + n:] == 7).all())
    xi = x.contiguous().clone()
    assert torch.equal(norm.layer_norm_fwd(xi, w, b, out=xi)[0], ref[0])
    _, mean, rstd = ref[:3]
    di = dy.contiguous().clone()
    assert torch.equal(norm.layer_norm_bwd(x.contiguous(), di, mean, rstd, w, out=di)[0], ref[3])


def test_without_parameters_and_empty():
    x, dy, w, b = make(6, 100, F32, F32)
    check(x, dy, None, None)
    check(x, dy, w, None)
    check(x, dy, None, None, eps=0.0)
    _, mean, rstd = norm.layer_norm_fwd(x, w, b)
    dx, dw, db = norm.layer_norm_bwd(x, dy, mean, rstd, w, need_params=False)
    assert dw is None and db is None
    assert torch.equal(dx, norm.layer_norm_bwd(x, dy, mean, rstd, w)[0])
    e = x[:0]
    y, mean, rstd = norm.layer_norm_fwd(e, w, b)
    assert y.shape == (0, 100) and mean.shape == (0,)
    dx, dw, db = norm.layer_norm_bwd(e, dy[:0], mean, rstd, w)
    assert dx.shape == (0, 100) and not dw.any() and not db.any() and dw.shape == (100,)
    z = torch.empty(4, 0, device=DEV)
    assert norm.layer_norm_fwd(z)[0].shape == (4, 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_constant_rows_large_offsets_and_non_finite_values(dtype):
    x, dy, w, b = make(9, 512, dtype, F32)
    x[2] = 3.0           # no variance: y = bias
    x[3] = x[3] * 0.001 + 100.0  # mean far from zero: centred squares
    y = check(x, dy, w, b)[0]
    assert torch.equal(y[2], b.to(dtype))
    ref = norm.layer_norm_fwd(x, w, b)
    bad = x.clone()
    bad[4, 100] = float("nan")
    bad[6, 511] = float("inf")
    y, mean, rstd = norm.layer_norm_fwd(bad, w, b)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], ref[0][keep]) and bool(torch.isnan(y[[4, 6]].float()).all())
    dx, _, _ = norm.layer_norm_bwd(bad, dy, mean, rstd, w)
    good = norm.layer_norm_bwd(x, dy, ref[1], ref[2], w)[0]
    assert torch.equal(dx[keep], good[keep]) and bool(torch.isnan(dx[[4, 6]].float()).all())


def test_gradient_against_differences():
    x, dy, w, b = make(5, 37, F32, F32)
    _, mean, rstd = norm.layer_norm_fwd(x, w, b)
    grads = norm.layer_norm_bwd(x, dy, mean, rstd, w)
    gen = torch.Generator().manual_seed(5)
    step = 2.0 ** -16
    for i, t in enumerate((x, w, b)):
        v = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        side = []
        for sgn in (1, -1):
            a = [o.f64(q) for q in (x, w, b)]
            a[i] = a[i] + sgn * step * v
            m = a[0].mean(1, keepdim=True)
            r = (((a[0] - m) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5
            side.append((((a[0] - m) * r * a[1] + a[2]) * o.f64(dy)).sum())
        diff = float((side[0] - side[1]) / (2 * step))
        # binary32 sums of 185 terms, and the differences' step^2.
        assert abs(diff - float((o.f64(grads[i]) * v).sum())) < 1e-4 * max(1.0, abs(diff))


def test_module_and_autograd():
    torch.manual_seed(0)
    m = norm.LayerNorm(96).to(DEV)
    with torch.no_grad():
        m.weight.add_(0.1 * torch.randn(96, device=DEV))
    x = torch.randn(4, 7, 96, device=DEV, dtype=BF16, requires_grad=True)
    y = m(x)
    dy = torch.randn_like(y)
    y.backward(dy)
    _, mean, rstd = norm.layer_norm_fwd(x.detach(), m.weight, m.bias)
    dx, dw, db = norm.layer_norm_bwd(x.detach(), dy, mean, rstd, m.weight.detach())
    assert torch.equal(x.grad, dx) and torch.equal(m.weight.grad, dw)
    assert torch.equal(m.bias.grad, db)
    m2 = norm.LayerNorm(96, bias=False).to(DEV)
    m2(x).sum().backward()
    assert m2.weight.grad is not None


def test_repeatable_streams_and_graph():
    x, dy, w, b = make(3000, 1024, BF16, F32)
    shared = dense.SharedBuffer()

    def step():
        y, mean, rstd = norm.layer_norm_fwd(x, w, b)
        return (y, *norm.layer_norm_bwd(x, dy, mean, rstd, w, shared=shared))

    ref = step()
    for a, c in zip(ref, step()):
        assert torch.equal(a, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(ref, got):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        x.copy_(torch.randn(3000, 1024, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, c in zip(got, step()):
            assert torch.equal(a, c), k
        torch.cuda.synchronize()


def test_refusals():
    x, dy, w, b = make(4, 64, F32, F32)
    _, mean, rstd = norm.layer_norm_fwd(x, w, b)
    with pytest.raises(TypeError):
        norm.layer_norm_fwd(x.half())
    with pytest.raises(TypeError):
        norm.layer_norm_fwd(x, w.half())
    with pytest.raises(TypeError):
        norm.layer_norm_fwd(x, w, b.to(BF16))
    with pytest.raises(ValueError):
        norm.layer_norm_fwd(x, w[:-1])
    with pytest.raises(ValueError):
        norm.layer_norm_fwd(x[0, 0])
    with pytest.raises(ValueError):
        norm.layer_norm_fwd(x, w.cpu())
    with pytest.raises(ValueError):
        norm.layer_norm_fwd(x, out=torch.empty(4, 63, device=DEV))
    with pytest.raises(TypeError):
        norm.layer_norm_fwd(x, out=torch.empty(4, 64, device=DEV, dtype=BF16))
    with pytest.raises(ValueError):
        norm.layer_norm_bwd(x, dy[:2], mean, rstd, w)
    with pytest.raises(ValueError):
        norm.layer_norm_bwd(x, dy, mean[:2], rstd, w)
    with pytest.raises(ValueError):
        norm.layer_norm_bwd(x, dy, mean, rstd.double(), w)
    with pytest.raises(mea.MeswishError):
        norm.layer_norm_fwd(x, w, b, eps=-1.0)
    flat = torch.randn(4 * 64 + 8, device=DEV)
    with pytest.raises(mea.MeswishError):  # a shifted output over its input
        norm.layer_norm_fwd(flat[:256].view(4, 64), w, b, out=flat[8:].view(4, 64))
