"""The parameters' step: AdamW over many tensors in one call, and the global norm
of their gradients.

Step count, learning rate and norm lie on the device and no call waits for it, so
a captured training step can end with the update: every replay counts a step and
reads the learning rate that it finds.
"""
from __future__ import annotations

import math
from operator import attrgetter

import numpy as np
import torch

from . import swin_attn as C
from .dropout import on

_C_DTYPE = {torch.bfloat16: C.SWIN_BF16, torch.float32: C.SWIN_F32}
_PARAM = np.dtype([(name, np.int64 if size == 8 else np.float32 if name == "decay" else np.int32) for name, size in
                   (("n", 8), ("dtype", 4), ("grad_dtype", 4), ("param", 8), ("master", 8), ("grad", 8), ("m", 8),
                    ("v", 8), ("m_scale", 8), ("v_scale", 8), ("decay", 4))], align=True)
UNIT = 256  # elements that share a scale of an 8-bit state


def _table(count):
    """A ctypes array of swin_attn_param, and its fields as numpy arrays."""
    entries = (C.swin_attn_param * max(count, 1))()
    return entries, np.frombuffer(entries, dtype=_PARAM, count=max(count, 1))


def _check_grad(name, g, shape, device):
    if not isinstance(g, torch.Tensor):
        raise ValueError("%s: expected a torch.Tensor, got %s" % (name, type(g).__name__))
    if g.device != device:
        raise ValueError("%s: on %s, expected %s" % (name, g.device, device))
    if g.dtype not in _C_DTYPE:
        raise ValueError("%s: dtype %s, expected bfloat16 or float32" % (name, g.dtype))
    if shape is not None and g.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(g.shape), tuple(shape)))
    if not g.is_contiguous():
        raise ValueError("%s: not contiguous" % name)


# Attributes of many tensors at once: a step's host path is a call for each of these, so they run without a
# frame of Python a tensor (183 tensors: the step's checks 180 us one by one, 60 us so).
_addresses, _sizes, _devices = (lambda ts, f=f: list(map(f, ts)) for f in (torch.Tensor.data_ptr, torch.Tensor.numel,
                                                                         torch.Tensor.get_device))
_dtype, _shape = attrgetter("dtype"), attrgetter("shape")


def _fit(tensors, device, shapes=None):
    """The C types of tensors that pass _check_grad; raises what it raises for the first that does not."""
    if set(map(type, tensors)) <= {torch.Tensor, torch.nn.Parameter}:
        types = list(map(_C_DTYPE.get, map(_dtype, tensors)))
        if (None not in types and set(_devices(tensors)) == {device.index} and all(map(torch.Tensor.is_contiguous, tensors))
                and (shapes is None or list(map(_shape, tensors)) == shapes)):
            return types
    for i, t in enumerate(tensors):
        _check_grad("tensors[%d]" % i, t, None if shapes is None else shapes[i], device)
    return [_C_DTYPE[t.dtype] for t in tensors]


def grad_norm(tensors, out=None, stream=None):
    """sqrt of the sum of all squares of bf16 or float32 tensors of one device, as a
    float32 tensor there (`out`, of one element, or a new one of no dimensions)."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("tensors: none given")
    dev = tensors[0].device if isinstance(tensors[0], torch.Tensor) else None
    if dev is None or dev.type != "cuda":
        raise ValueError("tensors[0]: expected a torch.Tensor on a CUDA device")
    types = _fit(tensors, dev)
    if out is not None and not (isinstance(out, torch.Tensor) and out.dtype == torch.float32 and out.device == dev
                                and out.numel() == 1):
        raise ValueError("out: want one float32 on %s" % (dev,))
    ctx = on(dev, stream)
    if ctx is not None:
        with ctx:
            return grad_norm(tensors, out)
    entries, at = _table(len(tensors))
    at["n"], at["grad_dtype"], at["grad"] = _sizes(tensors), types, _addresses(tensors)
    out = torch.empty((), dtype=torch.float32, device=dev) if out is None else out
    ws = torch.empty(C.swin_attn_adamw_workspace_bytes(), dtype=torch.uint8, device=dev)
    C.swin_attn_grad_norm(entries, len(tensors), out, ws)
    return out


class AdamW:
    """AdamW (decoupled weight decay) over all parameters at once.

    params: tensors, or dicts {"params": tensors, "weight_decay": d} for groups with
    a decay of their own. Parameters are contiguous float32 or bfloat16 tensors of
    one device, updated in place; a bfloat16 one is kept as the rounded copy of an
    fp32 master weight. state_bits: 32, or 8 (e4m3 with an fp32 scale of every 256
    values; 2 bytes an element instead of 8). max_norm: gradients are scaled down to
    this global norm where theirs is larger, and a step whose norm is not finite
    changes nothing and is not counted.

    On the device: `lr` (float32; write into it to change the learning rate),
    `steps` (int64: steps so far), `grad_norm` (float32, with max_norm: of
    the last step, before clipping). States lie in flat tensors, each parameter's
    from a multiple of 256 on: `m`, `v` (in 8 bits: e4m3, `v` holding the square
    roots, with `m_scale` and `v_scale`), `master` those of the bfloat16
    parameters, in order; a bfloat16 parameter that is written to otherwise is
    overwritten from its master by the next step.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32, max_norm=None):
        self.params, decays = [], []
        if isinstance(params, torch.Tensor):
            raise ValueError("params: a tensor, expected several (its rows are no parameters)")
        for group in params:
            some, decay = ([group], weight_decay) if not isinstance(group, dict) else (
                list(group["params"]), group.get("weight_decay", weight_decay))
            if not 0.0 <= decay < float("inf"):
                raise ValueError("weight_decay: at least 0 and finite, got %r" % (decay,))
            self.params += some
            decays += [float(decay)] * len(some)
        if not self.params:
            raise ValueError("params: none given")
        if not math.isfinite(lr):
            raise ValueError("lr: finite, got %r" % (lr,))
        if len(betas) != 2 or not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError("betas: two from 0 to below 1, got %r" % (betas,))
        if not 1e-30 <= eps < 1e30:
            raise ValueError("eps: positive and finite in fp32, got %r" % (eps,))
        if state_bits not in (8, 32):
            raise ValueError("state_bits: 32 or 8, got %r" % (state_bits,))
        if max_norm is not None and not 0.0 < max_norm < float("inf"):
            raise ValueError("max_norm: positive and finite, got %r" % (max_norm,))
        dev = self.params[0].device if isinstance(self.params[0], torch.Tensor) else None
        if dev is None or dev.type != "cuda":
            raise ValueError("params[0]: expected a torch.Tensor on a CUDA device")
        for i, p in enumerate(self.params):
            _check_grad("params[%d]" % i, p, None, dev)
        held = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()) for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(held, held[1:])):
            raise ValueError("params: two of them overlap, or one is given twice")
        self.device, self.betas, self.eps = dev, tuple(map(float, betas)), float(eps)
        self.state_bits, self.max_norm = state_bits, max_norm
        self._shapes = [p.shape for p in self.params]
        self._first, at, masters = [], 0, 0
        for p in self.params:
            self._first.append(at)
            at += -(-p.numel() // UNIT) * UNIT
            masters += -(-p.numel() // UNIT) * UNIT if p.dtype == torch.bfloat16 else 0
        state = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        with torch.cuda.device(dev), torch.no_grad():
            self._lr = torch.full((), float(lr), dtype=torch.float32, device=dev)
            self._steps = torch.zeros((), dtype=torch.int64, device=dev)
            self._grad_norm = None if max_norm is None else torch.zeros((), dtype=torch.float32, device=dev)
            self._m, self._v = (torch.zeros(at * state.itemsize, dtype=torch.uint8, device=dev).view(state) for _ in range(2))
            self._m_scale = self._v_scale = None
            if state_bits == 8:
                self._m_scale, self._v_scale = (torch.zeros(at // UNIT, dtype=torch.float32, device=dev) for _ in range(2))
            self._master = torch.zeros(masters, dtype=torch.float32, device=dev) if masters else None
            self._ws = torch.empty(C.swin_attn_adamw_workspace_bytes(), dtype=torch.uint8, device=dev)
            self._master_at, masters = [], 0
            for p in self.params:
                self._master_at.append(None)
                if p.dtype == torch.bfloat16 and p.numel():
                    self._master_at[-1] = masters
                    self.master[masters:masters + p.numel()].copy_(p.detach().reshape(-1))
                    masters += -(-p.numel() // UNIT) * UNIT
        # what does not change from step to step
        self._entries, self._at = _table(len(self.params))
        size = state_bits // 8
        a = self._at
        a["n"] = [p.numel() for p in self.params]
        a["dtype"] = [_C_DTYPE[p.dtype] for p in self.params]
        a["decay"] = decays
        a["master"] = [0 if o is None else self.master.data_ptr() + 4 * o for o in self._master_at]
        a["m"] = [self.m.data_ptr() + size * o for o in self._first]
        a["v"] = [self.v.data_ptr() + size * o for o in self._first]
        if state_bits == 8:
            a["m_scale"] = [self.m_scale.data_ptr() + 4 * (o // UNIT) for o in self._first]
            a["v_scale"] = [self.v_scale.data_ptr() + 4 * (o // UNIT) for o in self._first]
        # their memory stays with this object, so that an address that is unchanged is still theirs
        self._held, self._held_at = [p.detach() for p in self.params], [p.data_ptr() for p in self.params]
        a["param"] = self._held_at
        self._desc = C.swin_attn_adamw(*self.betas, self.eps, max_norm or 0.0, state_bits, self.lr.data_ptr(),
                                       self.steps.data_ptr(), None if max_norm is None else self.grad_norm.data_ptr())

    # their addresses are what the calls take: write into them, there is no other in their place
    lr, steps, grad_norm, m, v, m_scale, v_scale, master = (
        property(attrgetter("_" + n)) for n in ("lr", "steps", "grad_norm", "m", "v", "m_scale", "v_scale", "master"))

    def step(self, grads=None, stream=None):
        """One step with `grads` (one for each parameter, bfloat16 or float32, None: the parameter is left
        as it is), or with the parameters' own."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError("grads: %d for %d parameters" % (len(grads), len(self.params)))
        dev, there = self.device, [i for i, g in enumerate(grads) if g is not None]
        if not there:
            return
        if _addresses(self.params) != self._held_at:
            raise ValueError("params: one of them is not where it was (its data was replaced)")
        every = len(there) == len(grads)
        given = grads if every else [grads[i] for i in there]
        types = _fit(given, dev, self._shapes if every else [self._shapes[i] for i in there])
        ctx = on(dev, stream)
        if ctx is not None:
            with ctx:
                return self.step(grads)
        a = self._at
        if every:
            a["grad"], a["grad_dtype"] = _addresses(given), types
        else:
            a["grad"] = 0
            a["grad"][there], a["grad_dtype"][there] = _addresses(given), types
        C.swin_attn_adamw_step(self._desc, self._entries, len(grads), self._ws)
        # autograd reports what was saved before the step
        torch.autograd.graph.increment_version(self.params if every else [self.params[i] for i in there])

    def zero_grad(self):
        """Drop the parameters' gradients."""
        for p in self.params:
            p.grad = None

    def moments(self, i):
        """(m, v) of parameter i as the fp32 values that its states stand for."""
        p, o = self.params[i], self._first[i]
        m, v = (t[o:o + p.numel()].float() for t in (self.m, self.v))
        if self.state_bits == 8:
            u = slice(o // UNIT, o // UNIT - (-p.numel() // UNIT))
            m, v = (t * s[u].repeat_interleave(UNIT)[:p.numel()] for t, s in ((m, self.m_scale), (v, self.v_scale)))
            v = v * v
        return m.view(p.shape), v.view(p.shape)

    _STATE = ("lr", "steps", "m", "v", "m_scale", "v_scale", "master")

    def state_dict(self):
        """Copies of everything that a resumed run needs beside the parameters."""
        return {"state_bits": self.state_bits, "shapes": [tuple(s) for s in self._shapes],
                **{n: getattr(self, n).clone() for n in self._STATE if getattr(self, n) is not None}}

    def load_state_dict(self, state):
        """Take over a state_dict() of an AdamW over the same parameters and with the same state_bits."""
        if state.get("state_bits") != self.state_bits or state.get("shapes") != [tuple(s) for s in self._shapes]:
            raise ValueError("state: of other parameters or state_bits")
        for n in self._STATE:
            mine = getattr(self, n)
            if (mine is None) != (n not in state) or (mine is not None and mine.shape != state[n].shape):
                raise ValueError("state: %s does not fit" % n)
        for n in self._STATE:
            if getattr(self, n) is not None:
                getattr(self, n).copy_(state[n])
