"""Dropout from a counter-based generator: no mask is ever stored.

A decision is a pure function of (seed, step, site, index), so the backward
recomputes what the forward drew. The seed and the step live on the device in
a ``DropoutState``; the kernels read them when they run, so a captured step
replays with the step it finds there. A training step uses one state for all
its dropouts, each with a site of its own, and advances the state once its
backward is done.
"""
from __future__ import annotations

import torch

from . import swin_attn as C
from .autograd import once_differentiable, usable

_C_DTYPE = {torch.bfloat16: C.SWIN_BF16, torch.float32: C.SWIN_F32}


class DropoutState:
    """Seed (64 bits) and step of the generator, as an int64 CUDA tensor of two."""

    def __init__(self, seed, step=0, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if not 0 <= int(seed) < 2 ** 64:
            raise ValueError("seed: a whole number of 64 bits, got %r" % (seed,))
        seed = int(seed) - (2 ** 64 if int(seed) >= 2 ** 63 else 0)
        self._tensor = torch.tensor([seed, int(step)], dtype=torch.int64, device=device)

    @property
    def tensor(self):
        """The state itself (write into it to restore a saved one; dropouts keep its address)."""
        return self._tensor

    def advance(self, steps=1):
        """Go on to the next training step (on the current stream; may be
        captured). Between a forward and its backward it is an error, which
        autograd reports."""
        self.tensor[1:].add_(steps)


class Dropout:
    """One dropout of a model: its rate, its site and the state it draws from.

    The rate takes effect as T / 65536, T = round(rate * 65536); what is kept
    is scaled by 1 / (1 - T / 65536). Dropouts of one step need different
    sites, or they drop the same positions. None of the three changes later:
    for another rate (none, in an evaluation) pass another Dropout (or None).
    """

    def __init__(self, state, rate, site):
        if not isinstance(state, DropoutState):
            raise ValueError("state: expected a DropoutState, got %s" % type(state).__name__)
        if not (0.0 <= rate < 1.0) or round(rate * 65536) > 65535:
            raise ValueError("rate: from 0 to 65535/65536, got %r" % (rate,))
        if int(site) != site or not 0 <= site < 2 ** 32:
            raise ValueError("site: a whole number of 32 bits, got %r" % (site,))
        self._state, self._rate, self._site = state, float(rate), int(site)
        self.desc = C.swin_attn_drop(self._rate, self._site, state.tensor.data_ptr())

    state = property(lambda self: self._state)
    rate = property(lambda self: self._rate)
    site = property(lambda self: self._site)

    @property
    def active(self):
        return round(self._rate * 65536) > 0


def check_dropout(name, drop, device):
    if not isinstance(drop, Dropout):
        raise ValueError("%s: expected a Dropout, got %s" % (name, type(drop).__name__))
    if drop.state.tensor.device != device:
        raise ValueError("%s: its state is on %s, expected %s" % (name, drop.state.tensor.device, device))


def on(device, stream):
    """A context that makes `device` (and `stream`, if given) current while
    outputs are allocated and the call is issued, so that what the call
    allocates belongs to the stream that uses it; None where both are current."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream: on %s, the tensors are on %s" % (stream.device, device))
        return torch.cuda.stream(stream)
    return None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def same_rows(name, t, x):
    """`t` is like the checked tensor `x`: shape, type, device, contiguous, aligned."""
    if not (isinstance(t, torch.Tensor) and t.shape == x.shape and t.dtype == x.dtype and t.device == x.device
            and t.is_contiguous() and t.data_ptr() % 16 == 0):
        from .functional import check_tensor
        check_tensor(name, t, x.shape, x.dtype, x.device)  # raises, saying which


def apply_dropout(x, drop, span=1, out=None, stream=None):
    """y_i = x_i / kept where decision i // span keeps, else 0 (i: position in
    the contiguous x). span = 1: dropout; tokens * channels: whole images
    (stochastic depth). The backward is the same call on the gradient. `out`
    may be x. drop = None copies."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _C_DTYPE:
        raise ValueError("x: expected a bfloat16 or float32 torch.Tensor")
    if not x.is_cuda:
        raise ValueError("x: on %s, expected a CUDA device" % x.device)
    same_rows("x", x, x)
    if int(span) != span or span < 1:
        raise ValueError("span: at least 1, got %r" % (span,))
    if drop is not None:
        check_dropout("drop", drop, x.device)
    if out is not None:
        same_rows("out", out, x)
    span = min(int(span), 2 ** 62)  # from x's size on they are all the same
    ctx = on(x.device, stream)
    if ctx is not None:
        with ctx:
            return apply_dropout(x, drop, span, out)
    out = torch.empty_like(x) if out is None else out
    C.swin_attn_dropout(_C_DTYPE[x.dtype], x.numel(), span, x, drop.desc if drop else None, out)
    return out


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, drop, span):
        ctx.drop, ctx.span, ctx.linear = drop, span, True
        if drop is not None:
            ctx.save_for_backward(drop.state.tensor)  # a state advanced before the backward is reported
        return apply_dropout(usable(x), drop, span)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ctx.saved_tensors
        return apply_dropout(usable(dy), ctx.drop, ctx.span), None, None


def dropout(x, drop, span=1):
    """Autograd-aware dropout (see apply_dropout)."""
    return _DropoutFn.apply(x, drop, span)
