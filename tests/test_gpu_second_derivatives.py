"""The activations', the DenseNet stage's and the FFT convolution's gradients
cannot be differentiated again: under ``create_graph`` they are the same numbers,
and a second derivative raises instead of missing the kernels' terms."""

import pytest
import torch

import memory_efficient_activation_amd as mea
from memory_efficient_activation_amd import dense, fft

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(f, wrt, x):
    for loss in (lambda y: y.sum(), lambda y: y.pow(2).sum()):
        once = torch.autograd.grad(loss(f()), wrt)
        assert not any(g.requires_grad for g in once)
        graph = torch.autograd.grad(loss(f()), wrt, create_graph=True)
        for a, b in zip(once, graph):
            assert torch.equal(a, b)
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            (graph[0].pow(2).sum() + x.pow(3).sum()).backward()


@pytest.mark.parametrize("module", [mea.MemoryEfficientSwish(), mea.MemoryEfficientActivation("gelu")],
                         ids=["swish", "gelu"])
def test_activations(module):
    x = torch.randn(100, device=DEV, requires_grad=True)
    check(lambda: module(x), (x,), x)


def test_dense_stage():
    torch.manual_seed(0)
    stage = dense.EfficientBottleneckStage(12, 8, dense.SharedBuffer()).to(DEV)
    xs = [torch.randn(2, 6, 4, 4, device=DEV, requires_grad=True) for _ in range(2)]
    stats = [dense.bn_stats(x.detach()) for x in xs]
    torch.backends.cudnn.deterministic = True
    try:
        check(lambda: stage(xs, stats), (*xs, *stage.parameters()), xs[0])
    finally:
        torch.backends.cudnn.deterministic = False


def test_fft_convolution():
    torch.manual_seed(0)
    conv = fft.FFTConv2d(3, 4, 3).to(DEV)
    x = torch.randn(2, 3, 16, 16, device=DEV, requires_grad=True)
    check(lambda: conv(x), (x, conv.weight), x)
