"""What the library's autograd functions share."""
from __future__ import annotations

import functools

import torch
from torch.autograd import forward_ad


class _Gradient(torch.autograd.Function):
    """A gradient among what it was computed from: itself, with a backward that refuses."""

    @staticmethod
    def forward(ctx, grad, *sources):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the library's gradients have no gradient of their own: no second derivatives")


def first_order(backward):
    """For a Function's backward that calls the library: under create_graph=True its results refuse to be differentiated, by the
    incoming gradients, by what the forward pass saved and by ctx.sources, where it has set them (inputs that it need not save).
    The calls carry no graph, so a second derivative would lose their terms without a word wherever another path has one.
    (torch's once_differentiable looks at the incoming gradients alone, and lets those pass that need no gradient.)"""

    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        if not torch.is_grad_enabled():
            return backward(ctx, *grads)
        with torch.no_grad():
            results = backward(ctx, *grads)
        sources = [t for t in (*grads, *ctx.saved_tensors, *getattr(ctx, "sources", ())) if isinstance(t, torch.Tensor) and t.requires_grad]
        if not sources:
            return results
        return tuple(_Gradient.apply(r, *sources) if isinstance(r, torch.Tensor) else r for r in results)

    return wrapped


def no_tangents(what: str, *tensors) -> None:
    """For a call of the library outside an autograd function: raises where one of the tensors carries a forward-mode derivative, as
    such a function without a jvp does. requires_grad does not show it, and the library would drop it without a word."""
    if getattr(forward_ad, "_current_level", 0) < 0:   # no dual level is open (private to torch: asked for each tensor where it is missing)
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{what} has no forward-mode derivative")
