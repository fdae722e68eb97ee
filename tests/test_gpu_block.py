"""The blocks, which run the products, norms, units and borders together: against
the same formulas in binary64, with parts frozen, captured into graphs, on two
streams at once, and what they keep, to the byte."""

import pytest
import torch
import torch.nn.functional as F

from memory_efficient_activation_amd import block, dense, ffn_experiment as fx, linear, norm, residual

from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def act(kind, z):
    return {"swish": F.silu, "gelu": F.gelu, "tanh": torch.tanh}[kind](z)


def reference(m, p, x):
    """m's formula with the parameters p."""
    def ln(v, w, b, eps):
        return F.layer_norm(v, (v.shape[-1],), p[w], p[b], eps)

    def gated(n, at, kind):
        return (act(kind, n @ p[at + "w_gate"].t()) * (n @ p[at + "w_up"].t())) @ p[at + "w_down"].t()

    if isinstance(m, block.PreNormFeedForward):
        n = ln(x, "weight", "bias", m.eps)
        return x + F.linear(act(m.kind, F.linear(n, p["w1"], p.get("b1"))), p["w2"], p.get("b2"))
    if isinstance(m, block.GatedFeedForward):
        return gated(x, "", m.kind)
    n = ln(x, "norm.weight", "norm.bias", m.norm.eps)
    for i, (b, e) in enumerate(zip(m.blocks, m.borders)):
        z, at = gated(n, f"blocks.{i}.", b.kind), f"borders.{i}."
        if e.post:
            z = ln(z, at + "post_weight", at + "post_bias", e.eps)
        x = x + e.scale * p.get(at + "gate", 1.0) * z
        n = ln(x, at + "pre_weight", at + "pre_bias", e.eps)
    return n


MAKE = {
    "ungated": lambda d, h, t, s=None: block.PreNormFeedForward(d, h, shared=s, dtype=t),
    "ungated-plain": lambda d, h, t, s=None: block.PreNormFeedForward(d, h, "tanh", bias=False,
                                                                      shared=s, dtype=t),
    "gated": lambda d, h, t, s=None: block.GatedFeedForward(d, h, shared=s, dtype=t),
    "stack": lambda d, h, t, s=None: block.GatedFeedForwardStack(d, h, 2, gate=0.5, shared=s, dtype=t),
    "stack-sum": lambda d, h, t, s=None: block.GatedFeedForwardStack(d, h, 2, post=False, scale=0.5,
                                                                     shared=s, dtype=t),
}


def make(name, dim, hidden, dtype, shared=None, seed=0):
    torch.manual_seed(seed)
    m = MAKE[name](dim, hidden, dtype, shared).to(DEV)
    for p in m.parameters():  # ones and zeros hide what is forgotten
        p.data += 0.1 * torch.randn_like(p) * (1.0 if p.dim() == 1 else 0.0)
    return m


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", sorted(MAKE))
@pytest.mark.parametrize("lead,dim,hidden", [((1,), 64, 160), ((24,), 256, 520), ((3, 67), 200, 333),
                                             ((2, 300), 520, 1100)], ids=str)
def test_against_binary64(lead, dim, hidden, name, dtype):
    m = make(name, dim, hidden, dtype)
    x = torch.randn(*lead, dim, device=DEV).to(dtype).requires_grad_(True)
    dy = torch.randn(*lead, dim, device=DEV).to(dtype)
    y = m(x)
    got = [y, *torch.autograd.grad(y, (x, *m.parameters()), dy)]
    X = x.detach().cpu().double().requires_grad_(True)
    p = {k: v.detach().cpu().double().requires_grad_(True) for k, v in m.named_parameters()}
    Y = reference(m, p, X)
    want = [Y, *torch.autograd.grad(Y, (X, *p.values()), dy.cpu().double())]
    # About a dozen results on the way (a norm, two or three products, the
    # activation, a border, and back; twice that in a stack of two) are each off by
    # half a step of the type (bfloat16 2^-8) or, in binary32, by the activations'
    # 1e-5 and sums of up to 1100 terms (1100 2^-24 = 7e-5 of the terms' sizes), in
    # the norm of the whole.  A product by a random matrix carries a relative error
    # on by at most 1 + sqrt(k / m) < 3, and a random error by about 1; allowed is
    # that errors add up in size.  One token's gradients are single rows.
    steps = 24 if name.startswith("stack") else 12
    tol = steps * (2.0 ** -8 if dtype is BF16 else 8e-5)
    worst = 0.0
    for a, b in zip(got, want):
        a, b = a.detach().cpu().double(), b.detach()
        worst = max(worst, float((a - b).norm()) / float(b.norm()))
    say(f"[block] {name} {lead} {dim} {hidden} {dtype}: {worst:.3e} of {tol:.3e}")
    assert worst <= tol


def test_gradient_against_differences():
    """Along its own direction, for every parameter and the input, in binary32."""
    m = make("stack", 40, 72, F32)
    x = torch.randn(6, 40, device=DEV).requires_grad_(True)
    wrt = (x, *m.parameters())
    dy = torch.randn(6, 40, device=DEV)
    grads = torch.autograd.grad(m(x), wrt, dy)
    h = 2.0 ** -6

    def loss():
        return float((m(x).double() * dy.double()).sum())

    for t, g in zip(wrt, grads):
        size = float(g.norm())
        with torch.no_grad():
            before = t.clone()
            t += h / size * g
            up = loss()
            t.copy_(before - h / size * g)
            down = loss()
            t.copy_(before)
        # The loss is a sum of 240 terms, of sizes that add up to about 150, each
        # known to 1e-5: 1.5e-3 / h = 0.1 of the difference.  The third derivative
        # adds h^2 / 6 of itself, taken as 100 times the gradient.
        assert abs((up - down) / (2 * h) - size) <= 0.1 + 100 * h * h / 6 * size


@pytest.mark.parametrize("name", sorted(MAKE))
def test_frozen_parts(name):
    m = make(name, 72, 200, BF16, seed=5)
    x = torch.randn(3, 50, 72, device=DEV).to(BF16).requires_grad_(True)
    dy = torch.randn(3, 50, 72, device=DEV).to(BF16)
    tensors = dict(m.named_parameters(), x=x)
    want = dict(zip(tensors, torch.autograd.grad(m(x), list(tensors.values()), dy)))
    for wanted in ({k} for k in tensors):
        for k, t in tensors.items():
            t.requires_grad_(k in wanted)
        for k, g in zip(wanted, torch.autograd.grad(m(x), [tensors[k] for k in wanted], dy)):
            assert torch.equal(g, want[k]), k


@pytest.mark.parametrize("make_m", [lambda: linear.Linear(16, 24, "gelu"),
                                    lambda: block.PreNormFeedForward(16, 24),
                                    lambda: block.GatedFeedForwardStack(16, 24, 2, gate=0.5)],
                         ids=["Linear", "PreNormFeedForward", "GatedFeedForwardStack"])
def test_second_derivatives_raise(make_m):
    torch.manual_seed(3)
    m = make_m().to(DEV)
    x = torch.randn(5, 16, device=DEV, requires_grad=True)
    wrt = (x, *m.parameters())
    for loss in (lambda y: y.sum(), lambda y: y.pow(2).sum()):
        once = torch.autograd.grad(loss(m(x)), wrt)
        graph = torch.autograd.grad(loss(m(x)), wrt, create_graph=True)
        for a, b in zip(once, graph):
            assert torch.equal(a, b)
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            (graph[0].pow(2).sum() + x.pow(3).sum()).backward()


def test_no_tokens():
    for name in sorted(MAKE):
        m = make(name, 64, 96, F32)
        x = torch.zeros(2, 0, 64, device=DEV, requires_grad=True)
        y = m(x)
        grads = torch.autograd.grad(y, (x, *m.parameters()), torch.zeros_like(y))
        assert y.shape == x.shape and all(not bool(g.abs().any()) for g in grads[1:])


def capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = fn()
    return graph, outs


@pytest.mark.parametrize("tokens", [1, 24, 300])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_operators_in_graphs(tokens, dtype):
    """Two captured sequences of calls share one workspace; replays of both, in
    turn and after other work in the workspace, give the eager results."""
    shared = dense.SharedBuffer()
    gen = torch.Generator(device=DEV).manual_seed(7)

    def sequence(dim, units):
        x, z, dz, dn = (torch.randn(tokens, dim, device=DEV, generator=gen).to(dtype) for _ in range(4))
        w1 = (torch.randn(units, dim, device=DEV, generator=gen) * dim ** -0.5).to(dtype)
        w2 = (torch.randn(dim, units, device=DEV, generator=gen) * units ** -0.5).to(dtype)
        b1 = torch.randn(units, device=DEV, generator=gen).to(dtype)
        gate, pw, nw = (torch.randn(dim, device=DEV, generator=gen) for _ in range(3))

        def run():
            a = linear.linear_fwd(x, w1, b1, None, "gelu", shared=shared)
            s = linear.linear_fwd(a, w2, None, z, shared=shared)
            y, o, stats = residual.residual_norm_fwd(x, s, gate, (pw, None), (nw, None))
            g = residual.residual_norm_bwd(y, s, dz, dn, stats, gate, (pw, None), (nw, None),
                                           shared=shared)
            da, dw2, _ = linear.linear_bwd(a, w2, g.dz, shared=shared)
            dx, dw1, db1 = linear.linear_bwd(x, w1, da, b1, "gelu", shared=shared)
            return [a, s, y, o, g.dx, g.dz, g.dgate, g.dpost_weight, g.dpre_weight, da, dw2, dx, dw1,
                    db1]
        return run

    runs = [sequence(136, 333), sequence(256, 200)]
    want = [[t.clone() for t in run()] for run in runs]
    large = sequence(520, 1040)
    graphs = [capture(run) for run in runs]
    for k in range(3):
        for (graph, outs), expect in zip(graphs, want):
            for t in outs:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, expect)), k
        large()
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["ungated", "stack"])
def test_training_step_in_a_graph(name):
    """Forward and backward of the modules captured, no eager graph of their
    parameters alive."""
    m = make(name, 128, 264, BF16, dense.SharedBuffer(), seed=9)
    x = torch.randn(2, 75, 128, device=DEV).to(BF16).requires_grad_(True)
    dy = torch.randn(2, 75, 128, device=DEV).to(BF16)

    def run():
        y = m(x)
        return [y.detach(), *torch.autograd.grad(y, (x, *m.parameters()), dy)]

    want = [t.clone() for t in run()]
    graph, outs = capture(run)
    for k in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
        run()
        torch.cuda.synchronize()


def test_one_module_on_two_streams():
    m = make("stack", 104, 1000, BF16, seed=4)
    xs = [torch.randn(700, 104, device=DEV).to(BF16) for _ in range(2)]
    dys = [torch.randn(700, 104, device=DEV).to(BF16) for _ in range(2)]

    def step(k):
        x = xs[k].clone().requires_grad_(True)
        y = m(x)
        return (y.detach(), *torch.autograd.grad(y, (x, *m.parameters()), dys[k]))

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(step(k))
    torch.cuda.synchronize()
    for k in range(2):
        for res in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(res, want[k])), k


@pytest.mark.parametrize("dtype,es", [(F32, 4), (BF16, 2)])
@pytest.mark.parametrize("form", ["ungated", "stack"])
def test_what_the_blocks_keep(form, dtype, es):
    tokens, dim, hidden, blocks = 512, 256, 520, 3
    r = fx.measure(tokens, dim, hidden, blocks, dtype, reps=1, form=form)
    say(f"[block] {r}")
    if form == "ungated":  # each block's output, two binary32 values a token
        kept = blocks * tokens * (dim * es + 2 * 4)
    else:  # the first norm's rows and values; then z, the stream, its norm, four values
        kept = tokens * (dim * es + 2 * 4) + blocks * tokens * (3 * dim * es + 4 * 4)
    assert r["memory_efficient"]["retained_after_forward_bytes"] == kept
    # The plain blocks keep the activation's argument and result at the least.
    assert r["plain"]["retained_after_forward_bytes"] >= kept + blocks * tokens * hidden * es
    # As above, through three blocks.
    tol = 36 * (2.0 ** -8 if dtype is BF16 else 8e-5)
    assert r["memory_efficient"]["grad_rel_err_vs_f32"] <= tol


def test_the_shared_gradient_of_the_residual():
    """The residual and the input one tensor, used twice."""
    torch.manual_seed(2)
    m = linear.Linear(64, 64, "swish").to(DEV)
    x = torch.randn(40, 64, device=DEV, requires_grad=True)
    dy = torch.randn(40, 64, device=DEV)
    got = torch.autograd.grad(m(x, x), (x, m.weight, m.bias), dy)
    dx, dw, db = linear.linear_bwd(x.detach(), m.weight.detach(), dy, m.bias.detach(), "swish")
    assert torch.equal(got[0], dx + dy) and torch.equal(got[1], dw) and torch.equal(got[2], db)


def test_the_branch_and_the_stream_one_tensor():
    """z and x one tensor: the gradients of both add up."""
    torch.manual_seed(2)
    m = residual.ResidualNorm(72, gate=0.5).to(DEV)
    x = torch.randn(40, 72, device=DEV, requires_grad=True)
    d = [torch.randn(40, 72, device=DEV) for _ in range(2)]
    got = torch.autograd.grad(m(x, x), x, d)[0]
    a, b = x.detach().clone().requires_grad_(True), x.detach().clone().requires_grad_(True)
    da, db = torch.autograd.grad(m(a, b), (a, b), d)
    assert torch.equal(got, da + db)


def test_product_without_its_input():
    """The backward that no one's weight needs reads no input."""
    torch.manual_seed(6)
    for tokens, dim, units in ((1, 64, 96), (30, 100, 77), (300, 264, 320), (0, 64, 96)):
        for dtype in (F32, BF16):
            x = torch.randn(tokens, dim, device=DEV).to(dtype)
            w = torch.randn(units, dim, device=DEV).to(dtype)
            dy = torch.randn(tokens, units, device=DEV).to(dtype)
            want = linear.linear_bwd(x, w, dy, need_bias=True)
            got = linear.linear_bwd(None, w, dy, need_weight=False, need_bias=True)
            assert torch.equal(got[0], want[0]) and got[1] is None and torch.equal(got[2], want[2])


def test_norm_of_the_stack_is_the_layer_norm():
    torch.manual_seed(1)
    m = make("stack", 64, 96, F32)
    x = torch.randn(9, 64, device=DEV)
    n = norm.layer_norm_fwd(x, m.norm.weight.detach(), m.norm.bias.detach())[0]
    z = m.blocks[0](n)
    y, o = m.borders[0](x, z)
    rest = m.borders[1](y, m.blocks[1](o))[1]
    assert torch.equal(m(x), rest)
