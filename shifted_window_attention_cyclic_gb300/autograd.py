"""What the autograd functions of this package share."""
from __future__ import annotations

import functools

import torch


class _Refused(torch.autograd.Function):
    """Gradients as they are; their own derivative does not exist."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *dgrads):
        raise RuntimeError("gradients of gradients do not exist here: this backward is once_differentiable")


def once_differentiable(backward):
    """For a `backward` whose passes autograd cannot see into. Under
    create_graph its gradients depend on the incoming ones, and where
    `ctx.linear` is not set in the forward on the saved tensors too, whether or
    not the incoming ones carry a graph (torch's decorator of this name looks
    at those alone: of y.sum() they are constants, and the second term of
    f + |grad f|^2 would be left out without a word). Differentiating them
    raises."""

    @functools.wraps(backward)
    def wrapper(ctx, *dys):
        with torch.no_grad():
            grads = backward(ctx, *dys)
        constant = getattr(ctx, "linear", False) and not any(d is not None and d.requires_grad for d in dys)
        if constant or not torch.is_grad_enabled():
            return grads
        return _Refused.apply(torch.empty(0, requires_grad=True), *grads)

    return wrapper


def usable(t):
    """`t` as the library takes it, contiguous from a 16-byte boundary, or a copy that is (slices of larger tensors,
    and the gradients that a concatenation hands back, start anywhere)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t
