"""What stands around the attention of a block: the norm before it and the
residual join after it, with their gradients.

    h = N(x)                                              BlockNorm
    y = x + scale * gate * path * D(N_post(z)),  h = N_pre(y)     ResidualJoin

over [B, *grid, C] tensors. Each pass is one call into the CUDA library that
reads every activation once; the statistics are recomputed by the backward,
and dropout draws its decisions again, so nothing but the tensors themselves
is saved.
"""
from __future__ import annotations

import math
from collections import namedtuple

import torch

from . import swin_attn as C
from .autograd import once_differentiable, usable
from .dropout import check_dropout, on, same_rows
from .functional import _TORCH_DTYPE, check_tensor

_KINDS = {"none": C.SWIN_NORM_NONE, "layer": C.SWIN_NORM_LAYER, "rms": C.SWIN_NORM_RMS}

_NO_DROP = C.swin_attn_drop(0.0, 0, None)

JoinGrads = namedtuple("JoinGrads", "dx dz dpost_gamma dpost_beta dscale dgate dpre_gamma dpre_beta")


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_param(name, t, shape, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
    if t.shape != shape or t.dtype != torch.float32 or t.device != device or not t.is_contiguous():
        raise ValueError("%s: want a contiguous float32 %s on %s" % (name, tuple(shape), device))


class _Rows:
    """Channels and type of the rows, and the checks the calls share."""

    def __init__(self, channels, eps, dtype):
        if channels < 8 or channels % 8 or channels > 8192:
            raise ValueError("channels: a multiple of 8 up to 8192, got %r" % (channels,))
        if dtype not in _TORCH_DTYPE:
            raise ValueError("dtype: bf16 or f32, got %r" % (dtype,))
        if not 0.0 < eps < float("inf"):
            raise ValueError("eps: positive and finite, got %r" % (eps,))
        self.channels, self.eps, self.dtype = int(channels), float(eps), dtype
        self.torch_dtype = _TORCH_DTYPE[dtype]
        self.c_dtype = C.SWIN_BF16 if dtype == "bf16" else C.SWIN_F32

    def _rows(self, name, x):
        """Check the call's first tensor [B, *grid, C]; its descriptor."""
        if not isinstance(x, torch.Tensor):
            raise ValueError("%s: expected a torch.Tensor, got %s" % (name, type(x).__name__))
        if not x.is_cuda:
            raise ValueError("%s: on %s, expected a CUDA device" % (name, x.device))
        if x.dim() < 2 or x.shape[-1] != self.channels:
            raise ValueError("%s: shape %s, expected [B, *grid, %d]" % (name, tuple(x.shape), self.channels))
        if x.dtype != self.torch_dtype or not x.is_contiguous() or x.data_ptr() % 16:
            check_tensor(name, x, x.shape, self.torch_dtype, x.device)  # raises, saying which
        images, *grid = x.shape[:-1]
        return C.swin_attn_rows(images, math.prod(grid), self.channels, self.c_dtype)

    @staticmethod
    def _same(x, **tensors):
        for name, t in tensors.items():
            if t is not None:
                same_rows(name, t, x)

    @staticmethod
    def _workspace(rows, device, gated=False):
        """For parameter gradients; without a gate, that of the rows as one image."""
        if not gated:
            rows = C.swin_attn_rows(1, rows.images * rows.tokens, rows.channels, rows.dtype)
        return torch.empty(max(C.swin_attn_rows_workspace_bytes(rows), 256), dtype=torch.uint8, device=device)


class BlockNorm(_Rows):
    """The norm before a block, kind "layer" or "rms", of bf16 or f32 rows with
    float32 gamma and beta [C] (None: ones and zeros)."""

    def __init__(self, channels, kind="layer", eps=1e-5, dtype="bf16"):
        super().__init__(channels, eps, dtype)
        if kind not in ("layer", "rms"):
            raise ValueError("kind: layer or rms, got %r" % (kind,))
        self.kind = kind

    def _norm(self, x, gamma, beta):
        _check_param("gamma", gamma, (self.channels,), x.device)
        _check_param("beta", beta, (self.channels,), x.device)
        return C.swin_attn_norm(_KINDS[self.kind], self.eps, _addr(gamma), _addr(beta))

    def forward(self, x, gamma=None, beta=None, h=None, stream=None):
        """h = N(x); `h` may be x."""
        rows, norm = self._rows("x", x), self._norm(x, gamma, beta)
        self._same(x, h=h)
        ctx = on(x.device, stream)
        if ctx is not None:
            with ctx:
                return self.forward(x, gamma, beta, h)
        h = torch.empty_like(x) if h is None else h
        C.swin_attn_norm_fwd(rows, x, norm, h)
        return h

    def backward(self, x, dh, gamma=None, beta=None, dres=None, dx=None, want_params=True, stream=None):
        """(dx, dgamma, dbeta): dx = dres + N^T dh, where `dres` is the gradient
        that the residual path brings to x. dgamma and dbeta are None where
        gamma and beta are, or with want_params False."""
        rows, norm = self._rows("x", x), self._norm(x, gamma, beta)
        if dh is None:
            raise ValueError("dh: the backward needs the gradient of h")
        self._same(x, dh=dh, dres=dres, dx=dx)
        ctx = on(x.device, stream)
        if ctx is not None:
            with ctx:
                return self.backward(x, dh, gamma, beta, dres, dx, want_params)
        dx = torch.empty_like(x) if dx is None else dx
        dgamma = torch.empty_like(gamma) if want_params and gamma is not None else None
        dbeta = torch.empty_like(beta) if want_params and beta is not None else None
        ws = self._workspace(rows, x.device) if dgamma is not None or dbeta is not None else None
        C.swin_attn_norm_bwd(rows, x, norm, dh, dres, dx, dgamma, dbeta, ws)
        return dx, dgamma, dbeta


class ResidualJoin(_Rows):
    """The join after a block, fused with the next block's norm.

    post, pre: "none", "layer" or "rms". scale [C] (layer scale), gate [B, C]
    and the norms' gamma and beta [C] are float32, None where absent. drop
    (elements) and path (whole images: stochastic depth) are Dropouts.
    """

    def __init__(self, channels, post="none", pre="none", eps=1e-5, dtype="bf16"):
        super().__init__(channels, eps, dtype)
        for name, kind in (("post", post), ("pre", pre)):
            if kind not in _KINDS:
                raise ValueError("%s: none, layer or rms, got %r" % (name, kind))
        self.post, self.pre = post, pre

    def _join(self, x, post_gamma, post_beta, scale, gate, pre_gamma, pre_beta, drop, path):
        c, dev = (self.channels,), x.device
        for name, t, kind in (("post_gamma", post_gamma, self.post), ("post_beta", post_beta, self.post),
                              ("pre_gamma", pre_gamma, self.pre), ("pre_beta", pre_beta, self.pre)):
            if t is not None and kind == "none":
                raise ValueError("%s: the join has no such norm" % name)
            _check_param(name, t, c, dev)
        _check_param("scale", scale, c, dev)
        _check_param("gate", gate, (x.shape[0],) + c, dev)
        for name, d in (("drop", drop), ("path", path)):
            if d is not None:
                check_dropout(name, d, dev)
        return C.swin_attn_join(C.swin_attn_norm(_KINDS[self.post], self.eps, _addr(post_gamma), _addr(post_beta)),
                                C.swin_attn_norm(_KINDS[self.pre], self.eps, _addr(pre_gamma), _addr(pre_beta)),
                                _addr(scale), _addr(gate), drop.desc if drop else _NO_DROP, path.desc if path else _NO_DROP)

    def forward(self, x, z, post_gamma=None, post_beta=None, scale=None, gate=None, pre_gamma=None, pre_beta=None,
                drop=None, path=None, y=None, h=None, stream=None):
        """(y, h); h is None without a pre norm. `y` may be x or z."""
        rows = self._rows("x", x)
        if z is None:
            raise ValueError("z: the join needs the block's output")
        self._same(x, z=z, y=y, h=h)
        if h is not None and self.pre == "none":
            raise ValueError("h: the join has no pre norm")
        params = (post_gamma, post_beta, scale, gate, pre_gamma, pre_beta, drop, path)
        join = self._join(x, *params)
        ctx = on(x.device, stream)
        if ctx is not None:
            with ctx:
                return self.forward(x, z, *params, y, h)
        y = torch.empty_like(x) if y is None else y
        h = torch.empty_like(x) if h is None and self.pre != "none" else h
        C.swin_attn_join_fwd(rows, x, z, join, y, h)
        return y, h

    def backward(self, y, z, dy, dh=None, post_gamma=None, post_beta=None, scale=None, gate=None, pre_gamma=None,
                 pre_beta=None, drop=None, path=None, want_params=True, stream=None):
        """JoinGrads from the stored y (not x) and z. dy or dh may be None (no
        gradient reached it), not both. A parameter's gradient is None where
        the parameter is, or with want_params False."""
        rows = self._rows("y", y)
        if dy is None and dh is None:
            raise ValueError("dy, dh: at least one gradient is needed")
        if dh is not None and self.pre == "none":
            raise ValueError("dh: the join has no pre norm")
        if z is None:
            raise ValueError("z: the backward needs the block's output")
        self._same(y, z=z, dy=dy, dh=dh)
        params = (post_gamma, post_beta, scale, gate, pre_gamma, pre_beta)
        join = self._join(y, *params, drop, path)
        ctx = on(y.device, stream)
        if ctx is not None:
            with ctx:
                return self.backward(y, z, dy, dh, *params, drop, path, want_params)
        dx, dz = torch.empty_like(y), torch.empty_like(y)
        grads = [torch.empty_like(p) if want_params and p is not None else None for p in params]
        ws = self._workspace(rows, y.device, gate is not None) if any(g is not None for g in grads) else None
        C.swin_attn_join_bwd(rows, y, z, join, dy, dh, dx, dz, C.swin_attn_join_grads(*map(_addr, grads)), ws)
        return JoinGrads(dx, dz, *grads)


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, norm, x, gamma, beta):
        x = usable(x)
        ctx.norm = norm
        ctx.save_for_backward(x, gamma, beta)
        return norm.forward(x, gamma, beta)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, gamma, beta = ctx.saved_tensors
        want = any(ctx.needs_input_grad[2:])
        dx, dgamma, dbeta = ctx.norm.backward(x, usable(dh), gamma, beta, want_params=want)
        return None, dx, dgamma, dbeta


def block_norm(norm, x, gamma=None, beta=None):
    """Autograd-aware h = N(x) of a BlockNorm."""
    return _NormFn.apply(norm, x, gamma, beta)


class _JoinFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, join, x, z, post_gamma, post_beta, scale, gate, pre_gamma, pre_beta, drop, path):
        x, z = usable(x), usable(z)
        params = (post_gamma, post_beta, scale, gate, pre_gamma, pre_beta)
        y, h = join.forward(x, z, *params, drop=drop, path=path)
        ctx.join, ctx.drop, ctx.path = join, drop, path
        ctx.linear = join.post == join.pre == "none" and not any(ctx.needs_input_grad[3:9])
        ctx.set_materialize_grads(False)
        # the states are saved so that one advanced before the backward is reported
        ctx.save_for_backward(y, z, *params, *(d.state.tensor if d else None for d in (drop, path)))
        return (y, h) if h is not None else (y, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        y, z, *params = ctx.saved_tensors[:8]
        if dy is None and dh is None:
            return (None,) * 11
        dy, dh = (None if g is None else usable(g) for g in (dy, dh))
        g = ctx.join.backward(y, z, dy, dh, *params, drop=ctx.drop, path=ctx.path,
                              want_params=any(ctx.needs_input_grad[3:9]))
        return (None, *g, None, None)


def residual_join(join, x, z, post_gamma=None, post_beta=None, scale=None, gate=None, pre_gamma=None, pre_beta=None,
                  drop=None, path=None):
    """Autograd-aware join: (y, h), h None without a pre norm."""
    return _JoinFn.apply(join, x, z, post_gamma, post_beta, scale, gate, pre_gamma, pre_beta, drop, path)
