"""Memory that calls lend each other: it may be replaced by a larger block after
a graph was captured, or while another stream still works in it."""

import pytest
import torch

from memory_efficient_activation_amd import dense, ffn, fft, norm
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def unit(tokens, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = [torch.randn(*s, generator=gen, device=DEV) for s in
         ((tokens, 100), (300, 100), (300, 100), (tokens, 300))]
    return [v.to(BF16) for v in t]


def replays_after_growth(small, large, nbytes):
    """``small`` is captured, then ``large`` runs, and new tensors take what was
    freed: replays give the eager results and touch none of them."""
    want = [t.clone() for t in small()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        small()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = small()
    before = nbytes()
    large()
    assert nbytes() > before
    others = [torch.full((before,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    for k in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
        assert all(bool((t == 7).all()) for t in others), k
        large()
        torch.cuda.synchronize()
    say(f"replays equal to the eager result, {before} then {nbytes()} bytes lent")


def test_feed_forward_graph_after_growth():
    shared = dense.SharedBuffer()
    a, b = unit(400, 1), unit(4000, 2)

    def step(t):
        x, wg, wu, dh = t
        y, mean, rstd = norm.layer_norm_fwd(x)
        return (ffn.gated_ffn_fwd(y, wg, wu, shared=shared),
                *ffn.gated_ffn_bwd(y, wg, wu, dh, shared=shared),
                *norm.layer_norm_bwd(x, y, mean, rstd, shared=shared))

    replays_after_growth(lambda: step(a), lambda: step(b), lambda: shared.nbytes)


def test_fft_graph_after_growth():
    buf = fft.FrequencyBuffer()
    x, w = torch.randn(2, 3, 16, 16, device=DEV), torch.randn(4, 3, 3, 3, device=DEV)
    y = torch.randn(64, 3, 16, 16, device=DEV)
    replays_after_growth(lambda: [fft.fprop(x, w, buf)], lambda: [fft.fprop(y, w, buf)],
                         lambda: buf.nbytes)


@pytest.mark.parametrize("take", [lambda: dense.SharedBuffer().workspace,
                                  lambda: fft.FrequencyBuffer().get,
                                  lambda: (lambda b: lambda n, dev: b.view((n,), torch.uint8, dev))(
                                      dense.SharedBuffer())], ids=["workspace", "get", "view"])
def test_a_block_waits_for_the_stream_that_uses_it(take):
    """Replaced on another stream than its own, with that stream at work, a
    block's memory is not handed out before the work is done."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    take, size = take(), 64 << 20
    at = take(size, DEV).data_ptr()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert take(size, DEV).data_ptr() == at
        torch.cuda._sleep(200_000_000)
        done = torch.cuda.Event()
        done.record()
        take(2 * size, DEV)
    other = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert not done.query() and other.data_ptr() != at
    torch.cuda.synchronize()


def test_one_block_on_two_streams():
    """Forward and backward of one module on two streams at once, many times:
    each gives what it gives alone (to the roundings of the projection's library
    products, whose order of sums is not ours to know)."""
    torch.manual_seed(4)
    m = ffn.PreNormGatedFeedForward(104, 1000, dtype=BF16).to(DEV)
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
    for _ in range(20):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(step(k))
    torch.cuda.synchronize()
    for k in range(2):
        for res in got[k]:
            for a, b in zip(res, want[k]):
                a, b = a.float(), b.float()
                assert float((a - b).norm()) <= 2.0 ** -7 * float(b.norm()), k
