"""The border between blocks (norms, gate, scales, residual sum) on the GPU
against the binary64 oracle, within bounds that the oracle derives."""

import pytest
import torch

import memory_efficient_activation_amd as mea
from memory_efficient_activation_amd import dense, norm, residual
from oracle import ffn_oracle, finish_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(BF16, BF16), (F32, BF16), (F32, F32)]  # stream, branch
NORMS = [(True, True), (True, False), (False, True)]  # post, pre


def make(lead, n, types=(BF16, BF16), params=F32, norms=(True, True), gate=(), center=True, seed=0):
    """x, z, dy, do, and the arguments gate, post, pre."""
    rows = 1
    for s in lead:
        rows *= s
    gen = torch.Generator().manual_seed(seed + rows * 7919 + n * 131)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    x, z = ((normal(*lead, n) * (normal(n).abs() + 0.5) + normal(n) * 0.5).to(t).to(DEV)
            for t in types)
    dy, do = (normal(*lead, n).to(t).to(DEV) for t in types)

    def affine(on):
        if not on:
            return None
        w, b = (normal(n) * 0.25 + 1).to(params).to(DEV), (normal(n) * 0.25).to(params).to(DEV)
        return w, (b if center else None)

    g = None if gate is None else (normal(*gate, n) * 0.5 + 0.5).to(params).to(DEV)
    return x, z, dy, do, dict(gate=g, post=affine(norms[0]), pre=affine(norms[1]), center=center)


def present(values):
    return [v for v in values if v is not None]


def check(x, z, dy, do, args, scale=1.0, skip=1.0, eps=1e-5, shared=None):
    k = dict(args, scale=scale, skip=skip)
    y, out, stats = residual.residual_norm_fwd(x, z, eps=eps, **k)
    torch.cuda.synchronize()
    want, bound = o.border_forward(x, z, args["gate"], args["post"], args["pre"], scale, skip,
                                   args["center"], eps)
    got = present([y, out, *stats])
    assert len(got) == len(want)
    res = [ffn_oracle.worst(a, b, e) for a, b, e in zip(got, want, bound)]
    if args["pre"] is None:
        do = None
    grads = residual.residual_norm_bwd(y, z, dy, do, stats, shared=shared, **k)
    torch.cuda.synchronize()
    want, bound = o.border_backward(y, z, dy, do, stats, args["gate"], args["post"], args["pre"],
                                    scale, skip, args["center"])
    have = present(grads)
    assert len(have) == len(want)
    res += [ffn_oracle.worst(a, b, e) for a, b, e in zip(have, want, bound)]
    say(f"{tuple(x.shape)} {x.dtype} {z.dtype}: errors over bounds "
        + " ".join(f"{v:.3f}" for v in res))
    assert max(res) <= 1, res
    return y, out, stats, grads


WIDTHS = [1, 2, 7, 8, 9, 31, 32, 64, 65, 100, 256, 257, 512, 520, 1000, 1024, 1025, 2048, 2050,
          4095, 4096, 4104, 8192, 8193, 12000, 16384, 16385, 20000]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("n", WIDTHS)
def test_widths(n, types):
    check(*make((5,), n, types))
    check(*make((67,), n, types, params=types[1], center=False, seed=1), scale=0.25, skip=1.5)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("norms", NORMS, ids=str)
@pytest.mark.parametrize("gate", [None, (), (4,), (4, 30)], ids=str)
def test_parts_of_the_border(norms, gate, types):
    """Every combination of norms and gate (none, one, a sequence's, a row's)."""
    for n in (40, 200, 1500, 9000):
        for center in (True, False):
            check(*make((4, 30), n, types, BF16, norms, gate, center), scale=0.5)


@pytest.mark.parametrize("n", [24, 136, 700, 3000, 9000, 17000])
@pytest.mark.parametrize("lead,gate", [((1,), ()), ((1, 1), (1,)), ((300,), (300,)), ((3, 700), (3,)),
                                       ((700, 3), (700,)), ((2, 5, 7), (2, 5)), ((130, 33), (130,))],
                         ids=str)
def test_gate_rows(lead, gate, n):
    if n > 4000 and lead[0] * lead[-1] > 1000:
        lead = tuple(min(s, 30) for s in lead)
        gate = lead[:len(gate)]
    check(*make(lead, n, gate=gate))


def test_more_gate_rows_than_blocks():
    check(*make((1100, 5), 40, gate=(1100,)))
    check(*make((600, 70), 24, gate=(600,)))
    check(*make((520, 9), 2048, (F32, F32), gate=(520,)))
    check(*make((260, 40), 600, gate=(260,)))


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 511, 513, 4099])
def test_row_counts(rows, types):
    for n in (16, 264, 1024):
        check(*make((rows,), n, types), shared=dense.SharedBuffer())


def test_many_rows():
    check(*make((70000,), 24))
    check(*make((8, 2049), 1024, gate=(8,)), scale=0.3)


def test_parameters_left_out():
    x, z, dy, do, args = make((50,), 300, gate=None)
    w, b = args["post"]
    for post, pre in (((None, None), (None, None)), ((w, None), (None, b)), ((None, b), (w, b))):
        check(x, z, dy, do, dict(args, post=post, pre=pre))
    full = residual.residual_norm_fwd(x, z, **args)
    g = residual.residual_norm_bwd(full[0], z, dy, do, full[2], need_params=False, **args)
    h = residual.residual_norm_bwd(full[0], z, dy, do, full[2], **args)
    assert torch.equal(g.dx, h.dx) and torch.equal(g.dz, h.dz) and present(g[2:]) == []
    # No gradient of y: zeros.
    a = residual.residual_norm_bwd(full[0], z, None, do, full[2], **args)
    b = residual.residual_norm_bwd(full[0], z, torch.zeros_like(dy), do, full[2], **args)
    assert all(torch.equal(s, t) for s, t in zip(present(a), present(b)))


def test_statistics_are_layer_norms():
    """With neither gate nor post norm and z = 0, o is the layer normalization
    of x, and the statistics are its."""
    x, z, dy, do, args = make((33,), 777, (F32, F32), norms=(False, True), gate=None)
    y, out, stats = residual.residual_norm_fwd(x, torch.zeros_like(z), **args)
    ln, mean, rstd = norm.layer_norm_fwd(x, *args["pre"])
    assert torch.equal(y, x)
    for a, b in ((out, ln), (stats.pre_mean, mean), (stats.pre_rstd, rstd)):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("n", [40, 257, 1030, 9001])
def test_strides_and_alignment(n):
    x, z, dy, do, args = make((6, 11), n)
    ref = check(x, z, dy, do, args)

    def inside(t, left, right):
        big = torch.full((*t.shape[:-1], n + left + right), float("nan"), device=DEV, dtype=t.dtype)
        big[..., left:left + n] = t
        return big[..., left:left + n]

    for left, right in ((1, 2), (8, 8), (0, 3)):
        got = check(inside(x, left, right), inside(z, right, left), inside(dy, left, right),
                    inside(do, left, right), args)
        for a, b in zip(present([got[0], got[1], *got[2], *got[3]]),
                        present([ref[0], ref[1], *ref[2], *ref[3]])):
            assert torch.equal(a, b)
    wide = dy[:1].expand(6, 11, n)
    check(x, z, wide, do.transpose(0, 1).contiguous().transpose(0, 1), args)


def test_empty():
    for n in (16, 9000):
        for gate in (None, (), (0,)):
            x, z, dy, do, args = make((0,), n, gate=gate)
            y, out, stats = residual.residual_norm_fwd(x, z, **args)
            assert y.shape == (0, n) and out.shape == (0, n) and stats.pre_rstd.shape == (0,)
            g = residual.residual_norm_bwd(y, z, dy, do, stats, **args)
            assert all(not t.any() for t in present(g))
    x, z, dy, do, args = make((3, 0), 16, gate=(3,))
    y, out, stats = residual.residual_norm_fwd(x, z, **args)
    g = residual.residual_norm_bwd(y, z, dy, do, stats, **args)
    assert g.dgate.shape == (3, 16) and all(not t.any() for t in present(g))
    x, z, dy, do, args = make((3,), 0, gate=None)
    y, out, stats = residual.residual_norm_fwd(x, z, **args)
    assert y.shape == (3, 0)
    assert residual.residual_norm_bwd(y, z, dy, do, stats, **args).dx.shape == (3, 0)


@pytest.mark.parametrize("n", [33, 300, 2050, 9001, 17001])
def test_constant_and_non_finite_rows(n):
    x, z, dy, do, args = make((9,), n, (F32, F32))
    ref = residual.residual_norm_fwd(x, z, **args)
    rg = residual.residual_norm_bwd(ref[0], z, dy, do, ref[2], **args)
    for which in (x, z):
        t = which.clone()
        t[4] = float("nan")
        a, b = (t, z) if which is x else (x, t)
        y, out, stats = residual.residual_norm_fwd(a, b, **args)
        keep = [i for i in range(9) if i != 4]
        for got, want in ((y, ref[0]), (out, ref[1]), (stats.pre_rstd, ref[2].pre_rstd)):
            assert torch.equal(got[keep], want[keep]) and bool(torch.isnan(got[4]).all())
        g = residual.residual_norm_bwd(y, b, dy, do, stats, **args)
        assert torch.equal(g.dx[keep], rg.dx[keep]) and torch.equal(g.dz[keep], rg.dz[keep])
    # A constant row: the norm's result is its bias.
    z2 = z.clone()
    z2[2] = 3.0
    check(x, z2, dy, do, args)
    # Rows far from zero, and a mean times rstd past binary32: finite, as the
    # formulas are.
    z3 = z + 1000.0
    check(x, z3, dy, do, args)
    big = torch.full_like(z, 3e38)
    y, out, stats = residual.residual_norm_fwd(x, z, **args)
    stats = stats._replace(post_mean=torch.full_like(stats.post_mean, 3e38))
    g = residual.residual_norm_bwd(y, big, dy, do, stats, **args)
    assert all(bool(torch.isfinite(t.float()).all()) for t in present(g))


def test_repeats_bit_for_bit_and_streams():
    for n in (300, 4096, 9000):
        x, z, dy, do, args = make((8, 40), n, gate=(8,))

        def run():
            y, out, stats = residual.residual_norm_fwd(x, z, **args)
            return present([y, out, *stats, *residual.residual_norm_bwd(y, z, dy, do, stats, **args)])

        first = run()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = run()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for again in (run(), other):
            assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("post,pre", NORMS)
def test_autograd_and_module(post, pre, center):
    """Module and function against binary64 autograd of the definition."""
    torch.manual_seed(1)
    n = 72
    m = residual.ResidualNorm(n, post, pre, gate=0.5, scale=0.7, skip=1.2, center=center).to(DEV)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(torch.randn_like(p) * 0.3)
    x, z = (torch.randn(3, 11, n, device=DEV, requires_grad=True) for _ in range(2))
    dy, do = (torch.randn(3, 11, n, device=DEV) for _ in range(2))
    d = {k: v.detach().double().requires_grad_(True)
         for k, v in (("x", x), ("z", z), *m.named_parameters())}

    def norm64(v, name):
        if center:
            v = v - v.mean(-1, keepdim=True)
        v = v * ((v * v).mean(-1, keepdim=True) + m.eps) ** -0.5 * d[name + "_weight"]
        return v + d[name + "_bias"] if center else v

    p = norm64(d["z"], "post") if post else d["z"]
    y64 = m.skip * d["x"] + m.scale * d["gate"] * p
    loss = (y64 * dy.double()).sum()
    got = m(x, z)
    if pre:
        loss = loss + (norm64(y64, "pre") * do.double()).sum()
        torch.autograd.backward(got, (dy, do))
    else:
        got.backward(dy)
    loss.backward()
    for name, t in (("x", x), ("z", z), *m.named_parameters()):
        err = (t.grad.double() - d[name].grad).norm() / d[name].grad.norm()
        assert float(err) < 2e-6, (name, float(err))
    if pre:  # one of the two results alone
        x.grad = z.grad = None
        m(x, z)[1].backward(do)
        assert bool(torch.isfinite(x.grad).all())
        x.grad = None
        m(x, z)[0].backward(dy)
        assert torch.allclose(x.grad, m.skip * dy, rtol=1e-6)
    with pytest.raises(RuntimeError, match="differentiated again"):
        r = m(x, z)
        g, = torch.autograd.grad(r[0] if pre else r, z, dy, create_graph=True)
        g.sum().backward()


def test_refusals():
    x, z, dy, do, args = make((20,), 72)
    y, out, stats = residual.residual_norm_fwd(x, z, **args)
    fwd, bwd = residual.residual_norm_fwd, residual.residual_norm_bwd
    with pytest.raises(ValueError, match="at least one"):
        fwd(x, z)
    with pytest.raises(TypeError):
        fwd(x, z.float(), **args)
    with pytest.raises(TypeError):
        fwd(x.half(), z.half(), **args)
    with pytest.raises(ValueError):
        fwd(x, z[:19], **args)
    with pytest.raises(ValueError):
        fwd(x, z, **dict(args, gate=args["gate"][:71]))
    with pytest.raises(ValueError):
        fwd(x, z, **dict(args, gate=torch.ones(4, 72, device=DEV)))
    with pytest.raises(TypeError):
        fwd(x, z, **dict(args, gate=args["gate"].bfloat16()))
    with pytest.raises(ValueError):
        bwd(y, z, dy, None, stats, **args)
    with pytest.raises(ValueError):
        bwd(y, z, dy, do, residual.RowStats(None, None, None, None), **args)
    with pytest.raises(ValueError):
        bwd(y, z, dy.float(), do, stats, **args)
    with pytest.raises(mea.MeswishError):
        fwd(x, z, eps=float("nan"), **args)
    with pytest.raises(mea.MeswishError):
        fwd(x, z, scale=float("inf"), **args)
