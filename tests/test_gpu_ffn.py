"""The gated feed-forward unit on the GPU against the binary64 oracle, within
bounds that the oracle derives from the formulas and types."""

import pytest
import torch
import torch.nn.functional as F

import memory_efficient_activation_amd as mea
from memory_efficient_activation_amd import dense, ffn, norm
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
PARAM = {"swish": 1.0, "leaky_relu": 0.01}


def make(tokens, dim, hidden, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + tokens * 7919 + dim * 131 + hidden)
    s = max(dim, 1) ** -0.5
    t = [torch.randn(tokens, dim, generator=gen), torch.randn(hidden, dim, generator=gen) * s,
         torch.randn(hidden, dim, generator=gen) * s, torch.randn(tokens, hidden, generator=gen)]
    return [v.to(dtype).to(DEV) for v in t]


def check(x, wg, wu, dh, kind="swish", param=None, shared=None):
    p = PARAM.get(kind, 0.0) if param is None else param
    h = ffn.gated_ffn_fwd(x, wg, wu, kind, param, shared=shared)
    dx, dwg, dwu, h2 = ffn.gated_ffn_bwd(x, wg, wu, dh, kind, param, need_h=True, shared=shared)
    torch.cuda.synchronize()
    want, bound = o.ffn_forward(x, wg, wu, kind, p)
    res = [o.worst(h, want, bound), o.worst(h2, want, bound)]
    want, bound = o.ffn_backward(x, wg, wu, dh, kind, p)
    res += [o.worst(g, v, e) for g, v, e in zip((dx, dwg, dwu), want, bound)]
    say(f"{x.shape[0]} x {x.shape[-1]} -> {wg.shape[0]} {x.dtype} {kind}: errors over bounds "
        + " ".join(f"{r:.3f}" for r in res))
    assert max(res) <= 1, res
    return h, dx, dwg, dwu, h2


SHAPES = [(1, 1, 1), (1, 8, 8), (1, 64, 64), (1, 1024, 520), (2, 3, 5), (3, 100, 130),
          (8, 512, 64), (15, 96, 33), (16, 72, 200), (17, 72, 200), (24, 1000, 96),
          (31, 40, 512), (32, 512, 256), (33, 512, 256), (48, 264, 328), (64, 128, 96),
          (65, 136, 1000), (127, 64, 127), (128, 128, 64), (129, 72, 136), (200, 257, 131),
          (256, 256, 256), (257, 264, 520), (300, 512, 520), (513, 128, 384), (520, 1000, 264)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    check(*make(*shape, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", sorted(mea._lib.ACTS))
def test_activations(kind, dtype):
    for tokens in (1, 9, 200):
        x, wg, wu, dh = make(tokens, 96, 136, dtype, seed=3)
        x *= 3  # arguments out to where every activation is flat
        check(x, wg, wu, dh, kind)
    if kind in PARAM:
        check(*make(40, 64, 80, dtype), kind, 0.3)
        check(*make(5, 64, 80, dtype), kind, -0.7)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(768, 512, 768), (1024, 1024, 2048), (777, 1000, 2730),
                                   (1500, 136, 2056), (4099, 128, 256), (2048, 72, 512)], ids=str)
def test_larger_shapes(shape, dtype):
    check(*make(*shape, dtype), "gelu", shared=dense.SharedBuffer())


def test_many_tokens_few_units():
    check(*make(70000, 24, 40, BF16))
    check(*make(30000, 33, 17, F32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 256, 192), (20, 96, 72), (300, 264, 320)], ids=str)
def test_strides_and_alignment(shape, dtype):
    """Row distances and starts off every 16-byte boundary; leading
    dimensions; strided outputs whose neighbours stay as they were."""
    tokens, dim, hidden = shape
    x, wg, wu, dh = make(*shape, dtype)
    ref = check(x, wg, wu, dh)

    def inside(t, left, right):
        big = torch.full((t.shape[0], t.shape[1] + left + right), float("nan"), device=DEV,
                         dtype=t.dtype)
        big[:, left:left + t.shape[1]] = t
        return big[:, left:left + t.shape[1]]

    for l, r in ((1, 2), (8, 8), (0, 3)):
        got = check(inside(x, l, r), inside(wg, l, r), inside(wu, r, l), inside(dh, l, r))
        for a, c in zip(got, ref):
            assert torch.allclose(a.float(), c.float(), rtol=2 ** -7, atol=1e-2)
    x3 = x.view(tokens, 1, dim)
    assert torch.equal(ffn.gated_ffn_fwd(x3, wg, wu), ref[0].view(tokens, 1, hidden))
    for l, r in ((3, 4), (8, 0)):
        out = torch.full((tokens, hidden + l + r), 7.0, device=DEV, dtype=dtype)
        ffn.gated_ffn_fwd(x, wg, wu, out=out[:, l:l + hidden])
        assert torch.equal(out[:, l:l + hidden], ref[0])
        assert bool((out[:, :l] == 7).all()) and bool((out[:, l + hidden:] == 7).all())
    wt = wg.t().contiguous().t()  # k strided: copied
    assert torch.equal(ffn.gated_ffn_fwd(x, wt, wu), ref[0])


def test_empty_dimensions():
    for dtype in (F32, BF16):
        x, wg, wu, dh = make(0, 16, 24, dtype)
        assert ffn.gated_ffn_fwd(x, wg, wu).shape == (0, 24)
        dx, dwg, dwu = ffn.gated_ffn_bwd(x, wg, wu, dh)
        assert dx.shape == (0, 16) and dwg.shape == (24, 16) and not dwg.any() and not dwu.any()
        x, wg, wu, dh = make(5, 0, 24, dtype)
        assert not ffn.gated_ffn_fwd(x, wg, wu).any()
        dx, dwg, dwu = ffn.gated_ffn_bwd(x, wg, wu, dh, "sigmoid")
        assert dx.shape == (5, 0) and dwg.shape == (24, 0)
        x, wg, wu, dh = make(5, 16, 0, dtype)
        assert ffn.gated_ffn_fwd(x, wg, wu).shape == (5, 0)
        dx, dwg, dwu = ffn.gated_ffn_bwd(x, wg, wu, dh)
        assert dx.shape == (5, 16) and not dx.any() and dwg.shape == (0, 16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [5, 130, 300])
def test_non_finite_values_stay_in_their_rows(tokens, dtype):
    """A NaN or infinite token spoils its own rows, a unit's weight its own
    column; nothing leaks through the padding of tiles."""
    x, wg, wu, dh = make(tokens, 72, 136, dtype)
    ref = ffn.gated_ffn_fwd(x, wg, wu)
    rdx = ffn.gated_ffn_bwd(x, wg, wu, dh)[0]
    last = tokens - 1
    xb = x.clone()
    xb[last] = float("nan")
    got = ffn.gated_ffn_fwd(xb, wg, wu)
    assert torch.equal(got[:last], ref[:last]) and bool(torch.isnan(got[last].float()).all())
    assert torch.equal(ffn.gated_ffn_bwd(xb, wg, wu, dh)[0][:last], rdx[:last])
    wb = wg.clone()
    wb[135] = float("inf")
    got = ffn.gated_ffn_fwd(x, wb, wu)
    assert torch.equal(got[:, :135], ref[:, :135])
    # Only unit 135 of dWg and dWu can differ; dx is spoiled everywhere.
    a = ffn.gated_ffn_bwd(x, wg, wu, dh)
    c = ffn.gated_ffn_bwd(x, wb, wu, dh)
    assert torch.equal(a[1][:135], c[1][:135]) and torch.equal(a[2][:135], c[2][:135])


def test_values_past_the_type_become_infinite():
    x = torch.full((3, 64), 2.0 ** 100, device=DEV)
    w = torch.full((40, 64), 1.0, device=DEV)
    for dtype in (F32, BF16):
        h = ffn.gated_ffn_fwd(x.to(dtype), w.to(dtype), w.to(dtype))
        assert bool(torch.isinf(h.float()).all())


def test_only_what_is_needed():
    x, wg, wu, dh = make(50, 64, 72, BF16)
    dx, dwg, dwu = ffn.gated_ffn_bwd(x, wg, wu, dh)
    a = ffn.gated_ffn_bwd(x, wg, wu, dh, need_weights=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    a = ffn.gated_ffn_bwd(x, wg, wu, dh, need_x=False)
    assert a[0] is None and torch.equal(a[1], dwg) and torch.equal(a[2], dwu)


def test_gradient_against_differences():
    x, wg, wu, dh = make(7, 40, 24, F32)
    grads = ffn.gated_ffn_bwd(x, wg, wu, dh, "gelu")
    gen = torch.Generator().manual_seed(5)
    step = 2.0 ** -16
    for i, t in enumerate((x, wg, wu)):
        v = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        side = []
        for sgn in (1, -1):
            a = [o.f64(q) for q in (x, wg, wu)]
            a[i] = a[i] + sgn * step * v
            side.append((F.gelu(a[0] @ a[1].t()) * (a[0] @ a[2].t()) * o.f64(dh)).sum())
        diff = float((side[0] - side[1]) / (2 * step))
        # binary32 sums over at most 960 products, and the differences' step^2.
        assert abs(diff - float((o.f64(grads[i]) * v).sum())) < 1e-4 * max(1.0, abs(diff))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_runs_both_operators(dtype):
    """The pre-normalized block against the plain one in binary64; it keeps x,
    the statistics and nothing else."""
    torch.manual_seed(1)
    m = ffn.PreNormGatedFeedForward(96, 264, "swish", dtype=dtype).to(DEV)
    with torch.no_grad():
        m.weight.add_(0.1 * torch.randn(96, device=DEV))
        m.bias.add_(0.1 * torch.randn(96, device=DEV))
    x = torch.randn(3, 50, 96, device=DEV).to(dtype).requires_grad_(True)
    dy = torch.randn(3, 50, 96, device=DEV).to(dtype)
    m(x).backward(dy)  # workspaces grow
    for p in (x, *m.parameters()):
        p.grad = None
    base = torch.cuda.memory_stats()["requested_bytes.all.current"]
    y = m(x)
    kept = torch.cuda.memory_stats()["requested_bytes.all.current"] - base
    assert kept <= y.numel() * y.element_size() + 2 * 150 * 4, kept
    y.backward(dy)
    X, W, B, G, U, D = (o.f64(t).requires_grad_(True) for t in
                        (x, m.weight, m.bias, m.w_gate, m.w_up, m.w_down))
    n = F.layer_norm(X, (96,), W, B, m.eps)
    ref = X + (F.silu(n @ G.t()) * (n @ U.t())) @ D.t()
    grads = torch.autograd.grad(ref, (X, W, B, G, U, D), o.f64(dy))
    # Four roundings on the way (n, h, the projection, y; backward likewise):
    # each 2^-9 (2^-24 and 264-long binary32 sums) of the tensor's size.
    tol = 8 * 2.0 ** -9 if dtype == BF16 else 1e-5
    for a, c in zip((y, x.grad, m.weight.grad, m.bias.grad, m.w_gate.grad, m.w_up.grad,
                     m.w_down.grad), (ref.detach(), *grads)):
        a = o.f64(a)
        assert float((a - c).norm()) <= tol * float(c.norm())


def test_unit_module():
    torch.manual_seed(2)
    m = ffn.GatedUnit(64, 136, "gelu_tanh", dtype=BF16).to(DEV)
    x = torch.randn(5, 4, 64, device=DEV, dtype=BF16, requires_grad=True)
    h = m(x)
    dh = torch.randn_like(h)
    h.backward(dh)
    dx, dwg, dwu = ffn.gated_ffn_bwd(x.detach(), m.w_gate.detach(), m.w_up.detach(), dh,
                                     "gelu_tanh")
    assert torch.equal(x.grad, dx) and torch.equal(m.w_gate.grad, dwg)
    assert torch.equal(m.w_up.grad, dwu)


@pytest.mark.parametrize("shape", [(6, 512, 384), (400, 256, 512)], ids=str)
def test_repeatable_streams_and_graph(shape):
    x, wg, wu, dh = make(*shape, BF16)
    shared = dense.SharedBuffer()

    def step():
        return (ffn.gated_ffn_fwd(x, wg, wu, shared=shared),
                *ffn.gated_ffn_bwd(x, wg, wu, dh, shared=shared))

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
        x.copy_(torch.randn(x.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, c in zip(got, step()):
            assert torch.equal(a, c), k
        torch.cuda.synchronize()


def test_refusals():
    x, wg, wu, dh = make(4, 64, 72, F32)
    with pytest.raises(ValueError):
        ffn.gated_ffn_fwd(x, wg, wu, "softmax")
    with pytest.raises(TypeError):
        ffn.gated_ffn_fwd(x.half(), wg.half(), wu.half())
    with pytest.raises(TypeError):
        ffn.gated_ffn_fwd(x, wg.to(BF16), wu)
    with pytest.raises(ValueError):
        ffn.gated_ffn_fwd(x, wg[:, :-1], wu[:, :-1])
    with pytest.raises(ValueError):
        ffn.gated_ffn_fwd(x, wg, wu[:-1])
    with pytest.raises(RuntimeError):
        ffn.gated_ffn_fwd(x, wg.cpu(), wu)
    with pytest.raises(ValueError):
        ffn.gated_ffn_fwd(x, wg, wu, out=torch.empty(4, 71, device=DEV))
    with pytest.raises(ValueError):
        ffn.gated_ffn_bwd(x, wg, wu, dh[:, :-1])
    with pytest.raises(ValueError):
        ffn.gated_ffn_bwd(x, wg, wu, dh.to(BF16))
    with pytest.raises(mea.MeswishError):
        ffn.gated_ffn_fwd(x, wg, wu, "leaky_relu", float("nan"))
    with pytest.raises(mea.MeswishError):
        ffn.gated_ffn_fwd(x, wg, wu, "swish", 3e38)
    square = torch.randn(72, 72, device=DEV)
    with pytest.raises(mea.MeswishError):  # the output over a weight
        ffn.gated_ffn_fwd(square, square, wu.new_zeros(72, 72), out=square)
