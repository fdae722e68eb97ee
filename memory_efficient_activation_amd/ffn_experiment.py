"""Memory and time of a chain of transformer feed-forward blocks, plain
against memory-efficient.

The blocks' form is one of three, n = LN(x):

* gated: y = x + W_down (f(n Wg^T) * (n Wu^T)).  The plain block is eager
  PyTorch: autograd keeps, per token, the normalized row, both projections, the
  activation and the product beside the block's input.  The memory-efficient one
  (``ffn.PreNormGatedFeedForward``) keeps the input and two values and computes
  the rest again in the backward;
* ungated: y = x + W2 f(W1 n + b1) + b2 (``block.PreNormFeedForward``, which
  keeps the same);
* stack: gated blocks z = W_down (...) whose output is normalized and gated
  before it enters the stream, y = x + gate * LN(z), n = LN(y) the next block's
  input and the last one's result (``block.GatedFeedForwardStack``, which keeps
  y, z, n and four values).

The command runs one forward + backward of both on the same weights and
inputs (random), and prints one JSON line: bytes retained after the forward,
peak bytes over the step, the median step time, and how far the gradients of
each are from a plain block in binary32.

    python -m memory_efficient_activation_amd.ffn_experiment
    python -m memory_efficient_activation_amd.ffn_experiment --tokens 2048 --blocks 8 --dtype f32
    python -m memory_efficient_activation_amd.ffn_experiment --form stack
"""

from __future__ import annotations

import argparse
import json
import time

import torch
import torch.nn as nn
import torch.nn.functional as F

from .block import GatedFeedForwardStack, PreNormFeedForward
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


class PlainUngatedFeedForward(nn.Module):
    """The block without a gate in eager PyTorch."""

    def __init__(self, block: PreNormFeedForward):
        super().__init__()
        self.block = block

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        b = self.block
        n = F.layer_norm(x, (x.shape[-1],), b.weight, b.bias, b.eps)
        return x + F.linear(F.gelu(F.linear(n, b.w1, b.b1)), b.w2, b.b2)


class PlainStack(nn.Module):
    """The stack of gated blocks and their borders in eager PyTorch."""

    def __init__(self, stack: GatedFeedForwardStack):
        super().__init__()
        self.stack = stack

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        s, dim = self.stack, (x.shape[-1],)
        n = F.layer_norm(x, dim, s.norm.weight, s.norm.bias, s.norm.eps)
        for b, e in zip(s.blocks, s.borders):
            z = (F.silu(n @ b.w_gate.t()) * (n @ b.w_up.t())) @ b.w_down.t()
            x = x + e.scale * e.gate * F.layer_norm(z, dim, e.post_weight, e.post_bias, e.eps)
            n = F.layer_norm(x, dim, e.pre_weight, e.pre_bias, e.eps)
        return n


def chains(form: str, dim: int, hidden: int, blocks: int, dtype: torch.dtype):
    """(the memory-efficient chain, the plain one, which shares its parameters)."""
    shared = SharedBuffer()
    if form == "stack":
        stack = GatedFeedForwardStack(dim, hidden, blocks, gate=0.5, shared=shared, dtype=dtype)
        return stack.cuda(), PlainStack(stack)
    block, plain = {"gated": (PreNormGatedFeedForward, PlainFeedForward),
                    "ungated": (PreNormFeedForward, PlainUngatedFeedForward)}[form]
    efficient = nn.Sequential(*(block(dim, hidden, shared=shared, dtype=dtype)
                                for _ in range(blocks))).cuda()
    return efficient, nn.Sequential(*(plain(b) for b in efficient))


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
            dtype: torch.dtype = torch.bfloat16, reps: int = 5, form: str = "gated") -> dict:
    torch.manual_seed(0)
    efficient, plain = chains(form, dim, hidden, blocks, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, dim, device="cuda", generator=gen).to(dtype).requires_grad_(True)
    dy = torch.randn(tokens, dim, device="cuda", generator=gen).to(dtype)
    out = {"form": form, "tokens": tokens, "dim": dim, "hidden": hidden, "blocks": blocks,
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
    want = step(plain.float(), x.detach().float().requires_grad_(True), dy.float())[1]
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
    p.add_argument("--form", choices=["gated", "ungated", "stack"], default="gated")
    p.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = p.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    print(json.dumps(measure(a.tokens, a.dim, a.hidden, a.blocks, dtype, form=a.form)), flush=True)


if __name__ == "__main__":
    main()
