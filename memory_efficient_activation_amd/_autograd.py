"""What the package's autograd functions share."""

from __future__ import annotations

import functools

import torch


class _OnceOnly(torch.autograd.Function):
    """Its first ``count`` tensors as they are, depending on all of them;
    differentiating through it raises."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tensors[:count]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name}: its gradients come out of the library's kernels and "
                           "cannot be differentiated again")


def first_order(backward):
    """A function's ``backward`` whose results cannot be differentiated again.

    Autograd does not see into the kernels: under ``create_graph`` their
    results would count as constants, and a second derivative would silently
    miss their terms (also where the rest of the backward is torch's own).
    There the gradients depend on the inputs through a node that raises when
    it is differentiated; as numbers they are the same.  (Unlike torch's
    ``once_differentiable`` also where the upstream gradient is a constant.)
    """

    @functools.wraps(backward)
    def run(ctx, *upstream):
        if not torch.is_grad_enabled():
            return backward(ctx, *upstream)
        with torch.no_grad():
            grads = backward(ctx, *upstream)
        grads = grads if isinstance(grads, tuple) else (grads,)
        given = [g for g in grads if g is not None]
        sources = [t for t in (*upstream, *ctx.saved_tensors) if t is not None and t.requires_grad]
        if given and sources:
            name = type(ctx).__name__.removesuffix("Backward")
            given = list(_OnceOnly.apply(name, len(given), *given, *sources))
        return tuple(None if g is None else given.pop(0) for g in grads)

    return run
