"""What the library's autograd functions share."""
from __future__ import annotations

import functools

import torch


class _Gradient(torch.autograd.Function):
    """A gradient among what it was computed from: itself, with a backward that refuses."""

    @staticmethod
    def forward(ctx, grad, *sources):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the library's gradients have no gradient of their own: no second derivatives")


def first_order(backward):
    """For a Function's backward that calls the library: under create_graph=True its results refuse to be differentiated.
    The calls carry no graph, so a second derivative would lose their terms without a word wherever another path has one.
    (torch's once_differentiable looks at the incoming gradients alone, and lets those pass that need no gradient.)"""

    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        if not torch.is_grad_enabled():
            return backward(ctx, *grads)
        with torch.no_grad():
            results = backward(ctx, *grads)
        sources = [t for t in (*grads, *ctx.saved_tensors) if isinstance(t, torch.Tensor) and t.requires_grad]
        if not sources:
            return results
        return tuple(_Gradient.apply(r, *sources) if isinstance(r, torch.Tensor) else r for r in results)

    return wrapped
