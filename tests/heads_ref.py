"""64-bit reference of the head norm with rotary positions, in torch on the CPU,
written from the formulas. test_heads_ref_cpu.py holds its gradients against
central differences."""
from __future__ import annotations

from fractions import Fraction

import torch

from tests import rows_ref

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def turns(positions, frequencies, axis):
    """Angles [..., 1, pairs] of whole-number positions [..., axes], reduced exactly to one turn."""
    rows = positions.reshape(-1, positions.shape[-1]).tolist()
    out = []
    for row in rows:
        for f, a in zip(frequencies, axis):
            t = f * row[a]
            if abs(t) > 4:
                t = Fraction(f) * row[a]
                t = float(t - 2 * PI * round(t / (2 * PI)))
            out.append(t)
    return torch.tensor(out, dtype=torch.float64).view(positions.shape[:-1] + (1, len(frequencies)))


def grid_positions(images, grid):
    at = torch.stack(torch.meshgrid(*[torch.arange(g) for g in grid], indexing="ij"), -1)
    return at.view(1, -1, len(grid)).expand(images, -1, -1)


def rotate(u, t, layout, amplitude=1.0, back=False):
    """(turned u, what each value was summed from) of u [..., heads, hd] by t [..., 1, pairs]."""
    pairs = t.shape[-1]
    first = list(range(pairs)) if layout == "half" else list(range(0, 2 * pairs, 2))
    second = [i + pairs for i in first] if layout == "half" else [i + 1 for i in first]
    c, s = amplitude * torch.cos(t), amplitude * torch.sin(t) * (-1 if back else 1)
    a, b, out, size = u[..., first], u[..., second], u.clone(), u.abs()
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    size[..., first] = size[..., second] = abs(amplitude) * (a.abs() + b.abs())
    return out, size


def heads_fwd(x, t, layout, amplitude, kind, eps, gamma=None, beta=None):
    """(y, size) of x [images, tokens, heads, hd]; t None: nothing turns."""
    u = rows_ref.norm_fwd(x, kind, eps, gamma, beta)
    size = u.abs()
    if kind != "none":
        _, rstd = rows_ref.stats(x, kind, eps)
        g = 1.0 if gamma is None else gamma.abs()
        size = (x.abs() + x.abs().mean(-1, keepdim=True)) * rstd * g + (0.0 if beta is None else beta.abs())
    if t is None:
        return u, size
    y, _ = rotate(u, t, layout, amplitude)
    return y, rotate(size, torch.zeros_like(t), layout, amplitude)[1]


def heads_bwd(x, dy, t, layout, amplitude, kind, eps, gamma=None):
    """(dx, dgamma, dbeta) and the sizes of what each was summed from."""
    du, size = (dy, dy.abs()) if t is None else rotate(dy, t, layout, amplitude, back=True)
    if kind == "none":
        return (du, None, None), (size, None, None)
    dx, tg, tb, _ = rows_ref.norm_bwd(x, du, kind, eps, gamma)
    _, rstd = rows_ref.stats(x, kind, eps)
    spread = rows_ref.spread(x, kind, eps)
    g = size if gamma is None else size * gamma.abs()
    sx = rstd * spread * (g + g.mean(-1, keepdim=True) + spread * (g * spread).mean(-1, keepdim=True))
    return (dx, tg.sum((0, 1, 2)), tb.sum((0, 1, 2))), (sx, (size * spread).sum((0, 1, 2)), size.sum((0, 1, 2)))
