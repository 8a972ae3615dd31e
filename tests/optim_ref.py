"""64-bit reference of AdamW and of states in 8 bits, in torch on the CPU, written
from the formulas. test_optim_ref_cpu.py holds it against what defines it."""
from __future__ import annotations

import math

import torch

E4M3 = torch.tensor([0.0] + [k * 2.0**-9 for k in range(1, 8)]
                    + [(1 + k / 8) * 2.0**e for e in range(-6, 9) for k in range(8)][:-1], dtype=torch.float64)


def units(x):
    """[units, 256] with zeros behind the end."""
    n = -(-x.numel() // 256) * 256
    return torch.cat([x, x.new_zeros(n - x.numel())]).view(-1, 256)


def to_e4m3(x, floor=False):
    """(values, scales): nearest (ties to the even code) of x over its unit's largest magnitude / 448."""
    u = units(x)
    scale = u.abs().amax(1, keepdim=True) / 448
    r = torch.where(scale > 0, u / scale, 0.0)
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    up = torch.searchsorted(mid, r.abs().contiguous(), right=True)
    low = torch.searchsorted(mid, r.abs().contiguous(), right=False)
    code = torch.where(up == low, up, torch.where(up % 2 == 0, up, low))
    if floor:
        code = torch.where((r > 0) & (code == 0), 1, code)
    return (E4M3[code] * torch.sign(r)).view(-1)[:x.numel()], scale[:, 0]


def adamw(w, g, m, v, t, lr, decay, beta1, beta2, eps, clip=1.0):
    """(w, m, v) after step t (the first is 1)."""
    g = g * clip
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    step = lr / (1 - beta1**t) * m / (torch.sqrt(v) / math.sqrt(1 - beta2**t) + eps)
    return w * (1 - lr * decay) - step, m, v
