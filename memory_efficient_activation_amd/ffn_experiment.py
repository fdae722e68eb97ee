"""Memory and time of a chain of transformer feed-forward blocks, plain
against memory-efficient.

Each block is y = x + W_down (f(n Wg^T) * (n Wu^T)), n = LN(x).  The plain
block is eager PyTorch: autograd keeps, per token, the normalized row, both
projections, the activation and the product beside the block's input.  The
memory-efficient one (``ffn.PreNormGatedFeedForward``) keeps the input and
two values and computes the rest again in the backward.

The command runs one forward + backward of both on the same weights and
inputs (random), and prints one JSON line: bytes retained after the forward,
peak bytes over the step, the median step time, and how far the gradients of
each are from a plain block in binary32.

    python -m memory_efficient_activation_amd.ffn_experiment
    python -m memory_efficient_activation_amd.ffn_experiment --tokens 2048 --blocks 8 --dtype f32
"""

from __future__ import annotations

import argparse
import json
import time

import torch
import torch.nn as nn
import torch.nn.functional as F

from .dense import SharedBuffer
from .ffn import PreNormGatedFeedForward
from .memory_experiment import _requested


class PlainFeedForward(nn.Module):
    """The same block in eager PyTorch, sharing another block's parameters."""

    def __init__(self, block: PreNormGatedFeedForward):
        super().__init__()
        self.block = block

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        b = self.block
        n = F.layer_norm(x, (x.shape[-1],), b.weight, b.bias, b.eps)
        return x + (F.silu(n @ b.w_gate.t()) * (n @ b.w_up.t())) @ b.w_down.t()


def step(chain: nn.Module, x: torch.Tensor, dy: torch.Tensor):
    """One forward + backward; (bytes retained after the forward, gradients)."""
    for p in chain.parameters():
        p.grad = None
    base = _requested()
    y = chain(x)
    torch.cuda.synchronize()
    retained = _requested() - base
    y.backward(dy)
    return retained, [p.grad for p in chain.parameters()]


def measure(tokens: int = 16384, dim: int = 4096, hidden: int = 16384, blocks: int = 2,
            dtype: torch.dtype = torch.bfloat16, reps: int = 5) -> dict:
    torch.manual_seed(0)
    shared = SharedBuffer()
    efficient = nn.Sequential(*(PreNormGatedFeedForward(dim, hidden, shared=shared, dtype=dtype)
                                for _ in range(blocks))).cuda()
    plain = nn.Sequential(*(PlainFeedForward(b) for b in efficient))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, dim, device="cuda", generator=gen).to(dtype).requires_grad_(True)
    dy = torch.randn(tokens, dim, device="cuda", generator=gen).to(dtype)
    out = {"tokens": tokens, "dim": dim, "hidden": hidden, "blocks": blocks,
           "dtype": str(dtype).replace("torch.", "")}
    grads = {}
    for name, chain in (("plain", plain), ("memory_efficient", efficient)):
        step(chain, x, dy)  # workspaces and library plans
        for t in (x, *chain.parameters()):
            t.grad = None
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        base = _requested()
        retained, g = step(chain, x, dy)
        torch.cuda.synchronize()
        peak = _requested("peak") - base
        grads[name] = [t.float().clone() for t in g]
        times = []
        for _ in range(reps):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            step(chain, x, dy)
            torch.cuda.synchronize()
            times.append(time.perf_counter() - t0)
        out[name] = {"retained_after_forward_bytes": int(retained), "peak_step_bytes": int(peak),
                     "step_ms": round(1e3 * sorted(times)[len(times) // 2], 3)}
        x.grad = None
    ref = nn.Sequential(*(PlainFeedForward(b) for b in efficient)).float()
    want = step(ref, x.detach().float().requires_grad_(True), dy.float())[1]
    for name, g in grads.items():
        out[name]["grad_rel_err_vs_f32"] = max(float((a - b).norm() / b.norm())
                                               for a, b in zip(g, want))
    out["retained_ratio"] = round(out["plain"]["retained_after_forward_bytes"]
                                  / out["memory_efficient"]["retained_after_forward_bytes"], 3)
    return out


def main():
    p = argparse.ArgumentParser(description=__doc__,
                                formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=16384)
    p.add_argument("--dim", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=16384)
    p.add_argument("--blocks", type=int, default=2)
    p.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = p.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    print(json.dumps(measure(a.tokens, a.dim, a.hidden, a.blocks, dtype)), flush=True)


if __name__ == "__main__":
    main()
