"""Layer normalization and the gated unit at sizes that take the largest
tiles, and past 2^31 elements.  The reference is the oracle's binary64 on the
GPU (plain matrix products of binary64), whole or on sampled rows."""

import pytest
import torch

from memory_efficient_activation_amd import dense, ffn, norm
from oracle import ffn_oracle as o
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture
def on_gpu(monkeypatch):
    monkeypatch.setattr(o, "f64", lambda t: t.detach().to(torch.float64))


def make(tokens, dim, hidden, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    return (rnd(tokens, dim), rnd(hidden, dim, scale=dim ** -0.5),
            rnd(hidden, dim, scale=dim ** -0.5), rnd(tokens, hidden))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(4090, 4088, 2040), (4096, 2048, 4096), (1023, 2056, 6152),
                                   (8190, 264, 1000), (200, 8192, 6140), (200, 32760, 4090),
                                   (500, 1025, 16001), (8190, 200, 6140),
                                   (12280, 200, 16380)], ids=str)
def test_largest_tiles(shape, dtype, on_gpu):
    """The largest tiles, with edges inside tiles and vectors; in the last
    five shapes one product's sum is split over such tiles."""
    x, wg, wu, dh = make(*shape, dtype, 11)
    shared = dense.SharedBuffer()
    h = ffn.gated_ffn_fwd(x, wg, wu, shared=shared)
    dx, dwg, dwu, h2 = ffn.gated_ffn_bwd(x, wg, wu, dh, need_h=True, shared=shared)
    want, bound = o.ffn_forward(x, wg, wu, "swish", 1.0)
    res = [o.worst(h, want, bound), o.worst(h2, want, bound)]
    want, bound = o.ffn_backward(x, wg, wu, dh, "swish", 1.0)
    res += [o.worst(g, v, e) for g, v, e in zip((dx, dwg, dwu), want, bound)]
    say(f"{shape} {dtype}: errors over bounds " + " ".join(f"{r:.3f}" for r in res))
    assert max(res) <= 1, res


def test_unit_past_2_31_elements(on_gpu):
    """tokens x hidden of 2.3e9 elements: h, dh, the workspace and dx."""
    tokens, dim, hidden = 70001, 64, 32776
    x, wg, wu, _ = make(tokens, dim, hidden, BF16, 12)
    h = ffn.gated_ffn_fwd(x, wg, wu)
    rows = torch.tensor([0, 1, 255, 256, 32767, 65535, 65536, 69999, 70000], device=DEV)
    want, bound = o.ffn_forward(x[rows], wg, wu, "swish", 1.0)
    res = [o.worst(h[rows], want, bound)]
    dx, _, _, h2 = ffn.gated_ffn_bwd(x, wg, wu, h, need_weights=False, need_h=True)
    assert torch.equal(h2[rows], h[rows])
    want, bound = o.ffn_backward(x[rows], wg, wu, h[rows], "swish", 1.0)
    res.append(o.worst(dx[rows], want[0], bound[0]))
    say("errors over bounds " + " ".join(f"{r:.3f}" for r in res))
    assert max(res) <= 1, res


def test_norm_past_2_31_elements(on_gpu):
    rows, n = 530000, 4096  # 2.17e9 elements
    gen = torch.Generator(device=DEV).manual_seed(13)
    x = torch.empty(rows, n, device=DEV, dtype=BF16).normal_(generator=gen)
    w = torch.randn(n, generator=gen, device=DEV)
    y, mean, rstd = norm.layer_norm_fwd(x, w, w)
    some = torch.tensor([0, 1, 524287, 524288, 524289, 529998, 529999], device=DEV)
    want, bound = o.norm_forward(x[some], w, w, 1e-5)
    res = [o.worst(g[some], v, e) for g, v, e in zip((y, mean, rstd), want, bound)]
    dx, dw, db = norm.layer_norm_bwd(x, y, mean, rstd, w)
    want, bound = o.norm_backward(x[some], y[some], mean[some], rstd[some], w)
    res.append(o.worst(dx[some], want[0], bound[0]))
    # dweight and dbias over all rows, summed in binary64 a slice at a time.
    sw = torch.zeros(n, dtype=torch.float64, device=DEV)
    sb, aw, ab = sw.clone(), sw.clone(), sw.clone()
    for i in range(0, rows, 10000):
        d = y[i:i + 10000].double()
        t = d * ((x[i:i + 10000].double() - mean[i:i + 10000, None].double())
                 * rstd[i:i + 10000, None].double())
        sw += t.sum(0)
        sb += d.sum(0)
        aw += t.abs().sum(0)
        ab += d.abs().sum(0)
    depth = rows // 512 + 160
    res.append(o.worst(dw, sw, (depth + 4) * o.U * aw + o.half_unit(sw, F32) + o.TINY))
    res.append(o.worst(db, sb, depth * o.U * ab + o.half_unit(sb, F32) + o.TINY))
    say("errors over bounds " + " ".join(f"{r:.3f}" for r in res))
    assert max(res) <= 1, res
