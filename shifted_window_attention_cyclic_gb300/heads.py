"""What stands between the QKV projection and the attention: the norm of every
head and rotary positions, with their gradients.

    q, k, v = split(qkv);  q, k = R(N(q)), R(N(k))            AttentionHeads

The projection leaves [B, *grid, (heads + 2 kv_heads) * head_dim], the attention
takes contiguous q, k and v: one pass reads the packed tensor (or views of any
one row stride), norms and turns the heads of q and k, and writes all three where
the attention wants them; the backward goes the same way into one packed
gradient. The norms' statistics are recomputed, so nothing but the input is saved.
"""
from __future__ import annotations

import functools
import math
from collections import namedtuple
from fractions import Fraction

import numpy as np
import torch

from . import swin_attn as C
from .autograd import once_differentiable
from .dropout import on
from .functional import _TORCH_DTYPE
from .residual import _KINDS, _addr, _check_param

_LAYOUTS = {"half": C.SWIN_ROTARY_HALF, "interleaved": C.SWIN_ROTARY_INTERLEAVED}

HeadGrads = namedtuple("HeadGrads", "dq dk dv dq_gamma dq_beta dk_gamma dk_beta dqkv")


@functools.lru_cache(maxsize=None)
def _pi():
    """Pi to 2^-250 (Machin: 16 arctan(1/5) - 4 arctan(1/239))."""
    one = 1 << 260

    def arctan_inverse(n):
        term, total, k = one // n, 0, 0
        while term:
            total += (term if k % 2 == 0 else -term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total

    return Fraction(16 * arctan_inverse(5) - 4 * arctan_inverse(239), one)


class Rotary:
    """Rotary positions: the pairs of a head's first `dim` values turn by
    position * frequency.

    axes: position coordinates of a token (1: a sequence; 2 or 3: a grid). The
    pairs are shared out over the axes in order, pairs // axes each and one more
    for the last ones; an axis with n pairs has frequencies base^(-j / n).
    layout: "half" pairs value i with i + dim / 2, "interleaved" 2 i with 2 i + 1.
    scaling, for positions beyond those trained on, by `factor`:
      "linear"  positions divided by it (position interpolation);
      "ntk"     base * factor^(n / (n - 1)): the lowest frequency divided by it, the highest kept;
      "yarn"    by parts: frequencies that turn more than 32 times within `trained` positions are
                kept, those that turn less than once are divided by it, between them a ramp, and
                the turned values are scaled by 0.1 ln(factor) + 1 (Peng et al., "YaRN", 2023).
    Or give `frequencies` (radians a position, one a pair) with `axis_of` (each pair's axis) and
    `amplitude` (what turned values are multiplied by) outright.
    """

    def __init__(self, dim, axes=1, layout="half", base=10000.0, scaling=None, factor=1.0, trained=None,
                 frequencies=None, axis_of=None, amplitude=None):
        if int(dim) != dim or dim < 16 or dim % 16 or dim > 256:
            raise ValueError("dim: a multiple of 16 from 16 to 256, got %r" % (dim,))
        if axes not in (1, 2, 3):
            raise ValueError("axes: 1 to 3, got %r" % (axes,))
        if layout not in _LAYOUTS:
            raise ValueError("layout: half or interleaved, got %r" % (layout,))
        if scaling not in (None, "linear", "ntk", "yarn"):
            raise ValueError("scaling: linear, ntk, yarn or None, got %r" % (scaling,))
        if not (1.0 <= factor < float("inf")):
            raise ValueError("factor: at least 1 and finite, got %r" % (factor,))
        if scaling is None and factor != 1.0:
            raise ValueError("factor: without a scaling it has no use")
        if scaling == "yarn" and (trained is None or not trained > 0):
            raise ValueError("trained: yarn needs the positions trained on, got %r" % (trained,))
        if not (0.0 < base < float("inf")):
            raise ValueError("base: positive and finite, got %r" % (base,))
        pairs = dim // 2
        self.dim, self.axes, self.layout = int(dim), int(axes), layout
        if frequencies is None:
            if axis_of is not None:
                raise ValueError("axis_of: goes with frequencies")
            self.frequencies, self.axis_of = [], []
            for a in range(axes):
                n = pairs // axes + (1 if a >= axes - pairs % axes else 0)
                self.frequencies += self._axis(n, base, scaling, factor, trained)
                self.axis_of += [a] * n
        else:
            if scaling is not None:
                raise ValueError("scaling: frequencies are given outright")
            self.frequencies = [float(f) for f in frequencies]
            self.axis_of = [0] * pairs if axis_of is None and axes == 1 else list(axis_of or ())
            if len(self.frequencies) != pairs or len(self.axis_of) != pairs:
                raise ValueError("frequencies, axis_of: one for each of %d pairs, got %d and %d"
                                 % (pairs, len(self.frequencies), len(self.axis_of)))
            if not all(a in range(axes) for a in self.axis_of):
                raise ValueError("axis_of: axes from 0 to %d, got %r" % (axes - 1, self.axis_of))
            if not all(math.isfinite(f) for f in self.frequencies):
                raise ValueError("frequencies: finite, got %r" % (self.frequencies,))
        if amplitude is None:
            amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
        if not math.isfinite(amplitude):
            raise ValueError("amplitude: finite, got %r" % (amplitude,))
        self.amplitude = float(amplitude)
        # frequencies in turns a position, as 64-bit fixed point modulo one turn
        turn = 2 * _pi()
        self._freq = np.array([round(Fraction(f) / turn * 2 ** 64) % 2 ** 64 for f in self.frequencies], np.uint64)
        self._axis = np.array(self.axis_of, np.uint8)

    @staticmethod
    def _axis(n, base, scaling, factor, trained):
        if scaling == "ntk" and n > 1:
            base = base * factor ** (n / (n - 1))
        freq = [base ** (-j / n) for j in range(n)]
        if scaling == "linear":
            freq = [f / factor for f in freq]
        elif scaling == "yarn":
            kept = [min(1.0, max(0.0, (trained * f / (2 * math.pi) - 1) / 31)) for f in freq]
            freq = [f * ((1 - r) / factor + r) for f, r in zip(freq, kept)]
        return freq


class AttentionHeads:
    """Norm and rotary positions of the heads of q and k.

    heads (of q) and kv_heads (of k and v; as q's where not given) of head_dim
    values; rotary: a Rotary or None; norm: "none", "layer" or "rms" over every
    head's head_dim values, with float32 gamma and beta [head_dim] of q's heads and
    of k's (None: ones and zeros).

    q, k and v are [B, *grid, heads * head_dim] tensors, or views of one whose
    rows are evenly spaced (split() of a packed projection). Positions are a
    token's grid coordinates, or given as an int32 or int64 tensor
    [B, *grid, axes] or [*grid, axes] (without the last dimension where there is
    one axis).
    """

    def __init__(self, heads, head_dim, rotary=None, norm="none", eps=1e-5, dtype="bf16", kv_heads=None):
        if int(head_dim) != head_dim or head_dim < 16 or head_dim % 16 or head_dim > 256:
            raise ValueError("head_dim: a multiple of 16 from 16 to 256, got %r" % (head_dim,))
        for name, n in (("heads", heads), ("kv_heads", heads if kv_heads is None else kv_heads)):
            if int(n) != n or n < 1 or n * head_dim > 16384:
                raise ValueError("%s: at least 1, and %s * head_dim up to 16384, got %r" % (name, name, n))
        if rotary is not None and not isinstance(rotary, Rotary):
            raise ValueError("rotary: expected a Rotary, got %s" % type(rotary).__name__)
        if rotary is not None and rotary.dim > head_dim:
            raise ValueError("rotary: turns %d values, a head has %d" % (rotary.dim, head_dim))
        if norm not in _KINDS:
            raise ValueError("norm: none, layer or rms, got %r" % (norm,))
        if dtype not in _TORCH_DTYPE:
            raise ValueError("dtype: bf16 or f32, got %r" % (dtype,))
        if not 0.0 < eps < float("inf"):
            raise ValueError("eps: positive and finite, got %r" % (eps,))
        self.heads, self.kv_heads = int(heads), int(heads if kv_heads is None else kv_heads)
        self.head_dim, self.rotary, self.norm, self.eps, self.dtype = int(head_dim), rotary, norm, float(eps), dtype
        self.torch_dtype = _TORCH_DTYPE[dtype]
        self.q_width, self.kv_width = self.heads * self.head_dim, self.kv_heads * self.head_dim

    def split(self, qkv):
        """Views (q, k, v) of a packed [B, *grid, (heads + 2 kv_heads) * head_dim] tensor."""
        return qkv.split([self.q_width, self.kv_width, self.kv_width], -1)

    # -- what the calls share --
    def _stride(self, name, t, lead, width, device):
        """Elements from row to row of a checked tensor lead + (width,)."""
        if not isinstance(t, torch.Tensor):
            raise ValueError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
        if t.device != device or not t.is_cuda:
            raise ValueError("%s: on %s, expected %s" % (name, t.device, device if device.type == "cuda" else "a CUDA device"))
        if t.dtype != self.torch_dtype:
            raise ValueError("%s: dtype %s, expected %s" % (name, t.dtype, self.torch_dtype))
        if t.shape != lead + (width,):
            raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(lead + (width,))))
        stride = _row_stride(t)
        if stride is None:
            raise ValueError("%s: its rows are not evenly spaced, or their values not adjacent" % name)
        if t.data_ptr() % 16 or stride * t.element_size() % 16:
            raise ValueError("%s: rows do not start on 16-byte boundaries" % name)
        return stride

    def _describe(self, t, name, width, positions):
        """Leading dimensions of the call's first tensor, and the call's descriptor."""
        if not isinstance(t, torch.Tensor):
            raise ValueError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
        if t.dim() < 2:
            raise ValueError("%s: shape %s, expected [B, *grid, %d]" % (name, tuple(t.shape), width))
        lead = tuple(t.shape[:-1])
        grid, rot, tokens = lead[1:], self.rotary, math.prod(lead[1:])
        if max(lead[0], tokens) >= 2 ** 31 or lead[0] * tokens >= 2 ** 31:
            raise ValueError("%s: 2^31 rows or more" % name)
        d = C.swin_attn_heads(lead[0], 1, (tokens, 1, 1), self.head_dim,
                              C.SWIN_BF16 if self.dtype == "bf16" else C.SWIN_F32)
        if rot is None:
            if positions is not None:
                raise ValueError("positions: there is no rotary")
            return lead, d
        d.ndim = rot.axes
        d.rotary = C.swin_attn_rotary(rot.dim, _LAYOUTS[rot.layout], rot.amplitude, rot._freq.ctypes.data,
                                      rot._axis.ctypes.data)
        if positions is None:
            if len(grid) != rot.axes:
                raise ValueError("%s: %d grid dimensions, the rotary has %d axes (or give positions)"
                                 % (name, len(grid), rot.axes))
            for a, g in enumerate(grid):
                d.grid[a] = g
            return lead, d
        if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions: expected an int32 or int64 torch.Tensor")
        if positions.device != t.device:
            raise ValueError("positions: on %s, expected %s" % (positions.device, t.device))
        shape, one = tuple(positions.shape), rot.axes == 1
        if shape == lead + (rot.axes,) or (one and shape == lead):
            shared = 0
        elif shape == grid + (rot.axes,) or (one and shape == grid):
            shared = 1
        else:
            raise ValueError("positions: shape %s, expected %s or %s" % (shape, lead + (rot.axes,), grid + (rot.axes,)))
        if not positions.is_contiguous():
            raise ValueError("positions: not contiguous")
        d.rotary.position_bits = 32 if positions.dtype == torch.int32 else 64
        d.rotary.shared, d.rotary.positions = shared, positions.data_ptr()
        return lead, d

    def _norm(self, name, gamma, beta, device):
        if self.norm == "none" and (gamma is not None or beta is not None):
            raise ValueError("%s_gamma, %s_beta: the heads have no norm" % (name, name))
        _check_param(name + "_gamma", gamma, (self.head_dim,), device)
        _check_param(name + "_beta", beta, (self.head_dim,), device)
        return C.swin_attn_norm(_KINDS[self.norm], self.eps, _addr(gamma), _addr(beta))

    def forward(self, q, k=None, v=None, q_gamma=None, q_beta=None, k_gamma=None, k_beta=None, positions=None,
                q_out=None, k_out=None, v_out=None, stream=None):
        """(q, k, v) as the attention takes them, contiguous (v: copied; None where not given). An output
        may be its own input."""
        lead, d = self._describe(q, "q", self.q_width, positions)
        dev, parts = q.device, (C.swin_attn_head_part * 3)()
        if k is None and (k_gamma is not None or k_beta is not None):
            raise ValueError("k_gamma, k_beta: there is no k")
        given = [("q", q, q_out, self.q_width, q_gamma, q_beta), ("k", k, k_out, self.kv_width, k_gamma, k_beta),
                 ("v", v, v_out, self.kv_width, None, None)]
        count, todo = 0, []
        for name, x, out, width, gamma, beta in given:
            if x is None:
                if out is not None:
                    raise ValueError("%s_out: there is no %s" % (name, name))
                continue
            p = parts[count]
            p.heads, p.rotate = width // self.head_dim, int(name != "v" and self.rotary is not None)
            if name != "v":
                p.norm = self._norm(name, gamma, beta, dev)
            p.x, p.x_stride = x.data_ptr(), self._stride(name, x, lead, width, dev)
            if out is not None:
                p.out, p.out_stride = out.data_ptr(), self._stride(name + "_out", out, lead, width, dev)
            todo.append((p, name, width, out))
            count += 1
        ctx = on(dev, stream)
        if ctx is not None:
            with ctx:
                return self.forward(q, k, v, q_gamma, q_beta, k_gamma, k_beta, positions, q_out, k_out, v_out)
        got = dict.fromkeys("qkv")
        for p, name, width, out in todo:
            if out is None:
                out = torch.empty(lead + (width,), dtype=self.torch_dtype, device=dev)
                p.out, p.out_stride = out.data_ptr(), width
            got[name] = out
        C.swin_attn_heads_fwd(d, parts, count)
        return got["q"], got["k"], got["v"]

    def backward(self, dq, dk=None, dv=None, q=None, k=None, q_gamma=None, q_beta=None, k_gamma=None, k_beta=None,
                 positions=None, packed=False, want_params=True, stream=None):
        """HeadGrads from the gradients of the forward's outputs (dk, dv None where there was no k, v). q
        and k, the forward's inputs, are needed with a norm. packed: one tensor dqkv holds dq, dk and dv
        (which are views of it). A parameter's gradient is None where the parameter is, or with
        want_params False."""
        lead, d = self._describe(dq, "dq", self.q_width, positions)
        dev, parts = dq.device, (C.swin_attn_head_part * 3)()
        if packed and (dk is None or dv is None):
            raise ValueError("packed: needs dk and dv")
        if dk is None and (k_gamma is not None or k_beta is not None):
            raise ValueError("k_gamma, k_beta: there is no dk")
        given = [("q", q, dq, self.q_width, q_gamma, q_beta), ("k", k, dk, self.kv_width, k_gamma, k_beta),
                 ("v", None, dv, self.kv_width, None, None)]
        count, todo = 0, []
        for name, x, dy, width, gamma, beta in given:
            if dy is None:
                continue
            p = parts[count]
            p.heads, p.rotate = width // self.head_dim, int(name != "v" and self.rotary is not None)
            if name != "v":
                p.norm = self._norm(name, gamma, beta, dev)
                if self.norm != "none":
                    if x is None:
                        raise ValueError("%s: the backward of a norm needs its input" % name)
                    p.x, p.x_stride = x.data_ptr(), self._stride(name, x, lead, width, dev)
            p.dy, p.dy_stride = dy.data_ptr(), self._stride("d" + name, dy, lead, width, dev)
            todo.append((p, name, width, gamma, beta))
            count += 1
        ctx = on(dev, stream)
        if ctx is not None:
            with ctx:
                return self.backward(dq, dk, dv, q, k, q_gamma, q_beta, k_gamma, k_beta, positions, packed, want_params)
        got, at, dqkv = dict.fromkeys(HeadGrads._fields), 0, None
        if packed:
            dqkv = got["dqkv"] = torch.empty(lead + (self.q_width + 2 * self.kv_width,), dtype=self.torch_dtype, device=dev)
        for p, name, width, gamma, beta in todo:
            if packed:
                dx = dqkv[..., at:at + width]
                p.out_stride = dqkv.shape[-1]
                at += width
            else:
                dx = torch.empty(lead + (width,), dtype=self.torch_dtype, device=dev)
                p.out_stride = width
            got["d" + name], p.out = dx, dx.data_ptr()
            if want_params and gamma is not None:
                got["d%s_gamma" % name] = torch.empty_like(gamma)
                p.dgamma = got["d%s_gamma" % name].data_ptr()
            if want_params and beta is not None:
                got["d%s_beta" % name] = torch.empty_like(beta)
                p.dbeta = got["d%s_beta" % name].data_ptr()
        ws = None
        if any(got[n] is not None for n in ("dq_gamma", "dq_beta", "dk_gamma", "dk_beta")):
            ws = torch.empty(max(C.swin_attn_heads_workspace_bytes(d), 256), dtype=torch.uint8, device=dev)
        C.swin_attn_heads_bwd(d, parts, count, ws)
        return HeadGrads(**got)


def _row_stride(t):
    """Elements from row to row of [..., C], None where the rows are not evenly spaced."""
    if t.is_contiguous():
        return t.shape[-1]
    if t.stride(-1) != 1:
        return None
    stride = rows = None
    for size, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride, rows = s, size
        elif s != stride * rows:
            return None
        else:
            rows *= size
    return t.shape[-1] if stride is None else stride


def _usable(t):
    """`t` as the calls take it, or a contiguous copy that is."""
    if t is None:
        return None
    stride = _row_stride(t)
    if stride is not None and stride >= t.shape[-1] and t.data_ptr() % 16 == 0 and stride * t.element_size() % 16 == 0:
        return t
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class _HeadsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, heads, packed, qkv, k, v, q_gamma, q_beta, k_gamma, k_beta, positions):
        q, k, v = heads.split(qkv) if packed else (qkv, k, v)
        q, k, v = _usable(q), _usable(k), _usable(v)
        params = (q_gamma, q_beta, k_gamma, k_beta)
        out = heads.forward(q, k, v, *params, positions=positions)
        ctx.heads, ctx.packed, ctx.linear = heads, packed, heads.norm == "none"
        ctx.set_materialize_grads(False)
        some = heads.norm != "none"
        ctx.save_for_backward(q if some else None, k if some else None, *params, positions)
        ctx.shapes = [None if t is None else t.shape for t in out]
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, *douts):
        q, k, *params, positions = ctx.saved_tensors
        if all(d is None for d in douts):
            return (None,) * 10
        like = next(d for d in douts if d is not None)
        full = [None if s is None else like.new_zeros(s) if d is None else _usable(d) for s, d in zip(ctx.shapes, douts)]
        g = ctx.heads.backward(*full, q, k, *params, positions=positions, packed=ctx.packed,
                               want_params=any(ctx.needs_input_grad[5:9]))
        grads = (g.dqkv, None, None) if ctx.packed else (g.dq, g.dk, g.dv)
        return None, None, *grads, g.dq_gamma, g.dq_beta, g.dk_gamma, g.dk_beta, None


def attention_heads(heads, q, k=None, v=None, q_gamma=None, q_beta=None, k_gamma=None, k_beta=None, positions=None):
    """Autograd-aware AttentionHeads: (q, k, v) as the attention takes them."""
    return _HeadsFn.apply(heads, False, q, k, v, q_gamma, q_beta, k_gamma, k_beta, positions)


def attention_heads_packed(heads, qkv, q_gamma=None, q_beta=None, k_gamma=None, k_beta=None, positions=None):
    """The same from a projection's packed output, whose gradient comes back packed."""
    return _HeadsFn.apply(heads, True, qkv, None, None, q_gamma, q_beta, k_gamma, k_beta, positions)
