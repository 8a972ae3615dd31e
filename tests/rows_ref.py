"""64-bit references of the operators around the attention, in numpy and torch
on the CPU, written from the formulas: the dropout decisions, the norms, the
residual join and window attention with dropped probabilities. Gradients are
written out (not autograd); test_rows_ref_cpu.py holds them against central
differences."""
from __future__ import annotations

import numpy as np
import torch

M32 = np.uint64(0xFFFFFFFF)


def philox4x32(c0, c1, c2, c3, key, rounds):
    """Words [..., 4] (uint64 holding 32 bits) of the counters (arrays) under a 64-bit key."""
    c = [np.asarray(x, np.uint64) & M32 for x in np.broadcast_arrays(c0, c1, c2, c3)]
    for r in range(rounds):
        ka = np.uint64((key % 2**32 + r * 0x9E3779B9) % 2**32)
        kb = np.uint64((key // 2**32 + r * 0xBB67AE85) % 2**32)
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ ka, b & M32, (a >> np.uint64(32)) ^ c[3] ^ kb, a & M32]
    return np.stack(c, -1)


def threshold(rate):
    return int(np.rint(rate * 65536))


def kept_scale(rate):
    return 65536.0 / (65536 - threshold(rate))


def keep(index, seed, step, site, rate):
    """bool: does decision `index` (array of whole numbers) keep?"""
    index = np.asarray(index, np.uint64)
    block = index >> np.uint64(3)
    w = philox4x32(block & M32, block >> np.uint64(32), np.uint64(site), np.uint64(step % 2**32), seed, 7)
    e = (index & np.uint64(7)).astype(np.int64)
    word = np.take_along_axis(w, (e >> 1)[..., None], -1)[..., 0]
    half = np.where(e & 1, word >> np.uint64(16), word & np.uint64(0xFFFF))
    return half >= threshold(rate)


def weights(count, span, drop):
    """float64 [count]: 0 or the kept scale of each element; drop = (seed, step, site, rate) or None."""
    if drop is None or threshold(drop[3]) == 0:
        return np.ones(count)
    return keep(np.arange(count) // span, *drop) * kept_scale(drop[3])


# ---- norms and the join: x, z, ... float64 torch [B, T, C] ------------------
def stats(x, kind, eps):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    return mean, rstd


def spread(x, kind, eps):
    """1 + (|x| + mean |x|) / deviation: hat = (x - mean) rstd is off by the
    relative error of x, of the mean and of rstd times at most this, however
    small the difference x - mean itself is."""
    _, rstd = stats(x, kind, eps)
    return 1 + (x.abs() + x.abs().mean(-1, keepdim=True)) * rstd


def affine(hat, gamma, beta):
    out = hat if gamma is None else hat * gamma
    return out if beta is None else out + beta


def norm_fwd(x, kind, eps, gamma=None, beta=None):
    if kind == "none":
        return x
    mean, rstd = stats(x, kind, eps)
    return affine((x - mean) * rstd, gamma, beta)


def norm_bwd(x, dh, kind, eps, gamma=None):
    """(dx, dgamma terms, dbeta terms, size): terms unsummed; size bounds what dx is summed from."""
    mean, rstd = stats(x, kind, eps)
    hat = (x - mean) * rstd
    g = dh if gamma is None else dh * gamma
    c0 = g.mean(-1, keepdim=True) if kind == "layer" else 0.0
    c1 = (g * hat).mean(-1, keepdim=True)
    size = rstd * (g.abs() + g.abs().mean(-1, keepdim=True) + hat.abs() * (g * hat).abs().mean(-1, keepdim=True))
    return rstd * (g - c0 - hat * c1), dh * hat, dh, size


def join_weights(shape, scale, gate, drop, path):
    b, t, c = shape
    d = torch.from_numpy(weights(b * t * c, 1, drop)).view(b, t, c)
    p = torch.from_numpy(weights(b, 1, path)).view(b, 1, 1)
    s = torch.ones(c, dtype=torch.float64) if scale is None else scale
    g = torch.ones((b, 1, c), dtype=torch.float64) if gate is None else gate[:, None]
    return d, p, s, g


def join_fwd(x, z, post, pre, eps, par, drop, path, store=lambda y: y):
    d, p, s, g = join_weights(x.shape, par.get("scale"), par.get("gate"), drop, path)
    u = norm_fwd(z, post, eps, par.get("post_gamma"), par.get("post_beta"))
    y = x + s * g * p * d * u
    h = None if pre == "none" else norm_fwd(store(y), pre, eps, par.get("pre_gamma"), par.get("pre_beta"))
    return y, h


def join_bwd(y, z, dy, dh, post, pre, eps, par, drop, path):
    """{name: gradient} and {name: size}, size bounding the sums each was taken from."""
    d, p, s, g = join_weights(y.shape, par.get("scale"), par.get("gate"), drop, path)
    grad, size = {}, {}
    dx, sx = (torch.zeros_like(y), torch.zeros_like(y)) if dy is None else (dy, dy.abs())
    if pre != "none" and dh is not None:
        n, tg, tb, ns = norm_bwd(y, dh, pre, eps, par.get("pre_gamma"))
        dx, sx = dx + n, sx + ns
        for k, t, m in (("pre_gamma", tg, spread(y, pre, eps)), ("pre_beta", tb, 1.0)):
            grad["d" + k], size["d" + k] = t.sum((0, 1)), (dh.abs() * m).sum((0, 1))
    grad["dx"], size["dx"] = dx, sx
    w = p * d
    mean, rstd = stats(z, post, eps) if post != "none" else (0.0, 1.0)
    hat = (z - mean) * rstd
    u = affine(hat, par.get("post_gamma"), par.get("post_beta")) if post != "none" else z
    # what a sum over u is made of, term by term
    wide = spread(z, post, eps) if post != "none" else z.abs()
    ua = affine(wide, par.get("post_gamma"), None).abs() + (par["post_beta"].abs() if par.get("post_beta") is not None else 0.0)
    G, Ga = w * dx, w * sx
    du = s * g * G
    if post != "none":
        dz, tg, tb, ns = norm_bwd(z, du, post, eps, par.get("post_gamma"))
        gm = par.get("post_gamma")
        ka = Ga * (s * g).abs() if gm is None else Ga * (s * g * gm).abs()
        size["dz"] = rstd * (ka + ka.mean(-1, keepdim=True) + hat.abs() * (ka * hat.abs()).mean(-1, keepdim=True))
        for k, t, m in (("post_gamma", tg, wide), ("post_beta", tb, 1.0)):
            grad["d" + k], size["d" + k] = t.sum((0, 1)), (Ga * (s * g).abs() * m).sum((0, 1))
        grad["dz"] = dz
    else:
        grad["dz"], size["dz"] = du, Ga * (s * g).abs()
    grad["dscale"], size["dscale"] = (G * g * u).sum((0, 1)), (Ga * g.abs() * ua).sum((0, 1))
    grad["dgate"], size["dgate"] = (G * s * u).sum(1), (Ga * s.abs() * ua).sum(1)
    return grad, size


# ---- window attention with dropped probabilities ------------------------------
def attn(q, k, v, bias, land, tables, heads, drop, dout=None):
    """float64 [B, N, C] inputs, bias [rows, heads], land bool [B, N] or None, tables = (win_src, region, relidx)
    of one image. Returns o, lse [B, heads, N] and, with dout, dq, dk, dv, dbias."""
    src, region, rel = (torch.from_numpy(np.asarray(t).astype(np.int64)) for t in tables)
    b, tokens, c = q.shape
    hd, n = c // heads, src.shape[1]
    at, there = src.clamp(min=0), src >= 0
    cut = lambda x: x.view(b, tokens, heads, hd)[:, at].permute(0, 1, 3, 2, 4)  # noqa: E731

    def paste(x):
        out = torch.zeros((b, tokens, heads, hd), dtype=torch.float64)
        out[:, src[there]] = x.permute(0, 1, 3, 2, 4)[:, there]
        return out.view(b, tokens, c)

    Q, K, V = cut(q), cut(k), cut(v)
    live = there[None].expand(b, -1, -1)
    if land is not None:
        live = live & ~land[:, at]
    vis = live[:, :, :, None] & live[:, :, None, :] & (region[:, :, None] == region[:, None, :])
    s = Q @ K.transpose(-1, -2) / np.sqrt(hd) + bias[rel].permute(2, 0, 1)
    s = torch.where(vis[:, :, None], s, torch.full_like(s, -np.inf))
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))
    nb = -(-n // 8)
    row = (np.arange(b * heads).reshape(b, 1, heads, 1) * tokens + at.numpy()[None, :, None, :])[..., None]
    w = torch.ones_like(p)
    if drop is not None:
        w = torch.from_numpy(keep(row * (8 * nb) + np.arange(n), *drop) * kept_scale(drop[3]))
    lse_grid = torch.empty((b, heads, tokens), dtype=torch.float64)
    lse_grid[:, :, src[there]] = lse[..., 0].permute(0, 2, 1, 3)[:, :, there]
    out = {"o": paste((p * w) @ V), "lse": lse_grid}
    if dout is None:
        return out
    dO = cut(dout)
    dp = w * (dO @ V.transpose(-1, -2))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    out["dq"], out["dk"] = paste(ds @ K / np.sqrt(hd)), paste(ds.transpose(-1, -2) @ Q / np.sqrt(hd))
    out["dv"] = paste((p * w).transpose(-1, -2) @ dO)
    dbias = torch.zeros_like(bias)
    dbias.index_add_(0, rel.flatten(), ds.sum((0, 1)).flatten(1).t())
    out["dbias"] = dbias
    return out
