"""Reference values and error bounds of window attention with dropped
probabilities, per output element, from the 64-bit matrices of all window
pairs. (Written for the dBias of head_dim 128 with O given and for rates that
drop nearly everything, where one bar for a whole tensor catches nothing.)"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from shifted_window_attention_cyclic_gb300 import workloads
from tests import rows_ref as ref
from tests.parity_util import problem_of

HALF = 2.0**-8  # half a step of bf16, relative
E32 = 2.0**-24  # of fp32


class Pairs:
    """All pairs of a case's windows, [B, windows, heads, n, n] or [..., n, hd], in float64."""

    def __init__(self, case, rate, seed, step, site, seed_index=700):
        grid, window, shift, periodic, heads, hd, batch, dtype, land_p = case
        wl = workloads.custom(grid, window, shift, periodic, heads, hd, batch, dtype, land_p, seed_index=seed_index)
        x = workloads.generate(wl)
        src, region, _, rel = oracle.tables(problem_of(wl))
        src, region, self.rel = (torch.from_numpy(np.asarray(t).astype(np.int64)) for t in (src, region, rel))
        self.src, self.heads, self.hd, self.dtype, self.c = src, heads, hd, dtype, ref.kept_scale(rate)
        self.bias = torch.from_numpy(x["bias"]).double()
        self.batch, self.tokens, n = batch, int(np.prod(grid)), src.shape[1]
        at, self.there = src.clamp(min=0), src >= 0
        self.Q, self.K, self.V, self.dO = (
            torch.from_numpy(x[t]).double().view(batch, self.tokens, heads, hd)[:, at].permute(0, 1, 3, 2, 4)
            for t in ("q", "k", "v", "dout"))
        live = self.there[None].expand(batch, -1, -1)
        if x["land"] is not None:
            live = live & (torch.from_numpy(x["land"]).view(batch, -1) == 0)[:, at]
        self.visible = (live[:, :, :, None] & live[:, :, None, :] & (region[:, :, None] == region[:, None, :]))[:, :, None]
        s = self.Q @ self.K.transpose(-1, -2) / hd**0.5 + self.bias[self.rel].permute(2, 0, 1)
        s = torch.where(self.visible, s, torch.full_like(s, -np.inf))
        lse = torch.logsumexp(s, -1, keepdim=True)
        self.p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))
        row = (np.arange(batch * heads).reshape(batch, 1, heads, 1) * self.tokens + at.numpy()[None, :, None, :])[..., None]
        self.keep = torch.from_numpy(ref.keep(row * (8 * -(-n // 8)) + np.arange(n), seed, step, site, rate)).double()
        self.w = self.keep * self.c
        # relative error of a probability in fp32: its score's, the row maximum's and the sum's, an exponential and a
        # quotient (a score sums hd products; scores enter as themselves and in the row's sum)
        s_err = (hd + 8) * E32 * (self.Q.abs() @ self.K.abs().transpose(-1, -2) / hd**0.5 + 8)
        self.e_p = 2 * torch.where(self.visible, s_err, torch.zeros_like(s_err)).amax() + (n + 16) * E32

    def grid(self, x):
        """[B, windows, heads, n, hd] -> [B, tokens, heads * hd]."""
        out = torch.zeros((self.batch, self.tokens, self.heads, self.hd), dtype=torch.float64)
        out[:, self.src[self.there]] = x.permute(0, 1, 3, 2, 4)[:, self.there]
        return out.view(self.batch, self.tokens, -1)

    def rows(self, x):
        """[B, windows, heads, n, n] summed into bias rows [rows, heads]."""
        return torch.zeros_like(self.bias).index_add_(0, self.rel.flatten(), x.sum((0, 1)).flatten(1).t())

    def ds(self, scale=None):
        """dS, with the kept scale replaced by `scale` (a planted mistake) or as it is."""
        w = self.w if scale is None else self.keep * scale
        dp = w * (self.dO @ self.V.transpose(-1, -2))
        return self.p * (dp - (self.p * dp).sum(-1, keepdim=True))

    def outputs(self, scale=None):
        w, ds = self.w if scale is None else self.keep * scale, self.ds(scale)
        r = self.hd**-0.5
        return {"o": self.grid((self.p * w) @ self.V), "dv": self.grid((self.p * w).transpose(-1, -2) @ self.dO),
                "dq": self.grid(ds @ self.K * r), "dk": self.grid(ds.transpose(-1, -2) @ self.Q * r), "dbias": self.rows(ds)}

    def bounds(self):
        """{name: bound} of each element's error: the sum of its terms' absolute values times their relative errors.
        P and dS are rounded to bf16 where the tensor cores read them, outputs where they are stored; dBias sums fp32
        dS. dP is a sum of hd products, delta one of n pairs; every sum is fp32."""
        n = self.p.shape[-1]
        half, store = (HALF, HALF) if self.dtype == "bf16" else (0.0, E32)
        pa = self.p * self.w
        dpa = self.w * (self.dO.abs() @ self.V.abs().transpose(-1, -2))
        dsa = self.p * (dpa + (self.p * dpa).sum(-1, keepdim=True))
        e_ds = 2 * self.e_p + (self.hd + 2 * n + 16) * E32
        e_sum = (2 * n + 16) * E32
        r = self.hd**-0.5
        want = self.outputs()
        size = {"o": self.grid(pa @ self.V.abs()), "dv": self.grid(pa.transpose(-1, -2) @ self.dO.abs()),
                "dq": self.grid(dsa @ self.K.abs() * r), "dk": self.grid(dsa.transpose(-1, -2) @ self.Q.abs() * r)}
        out = {name: (1 + store) * ((1 + half) * (1 + (self.e_p if name in ("o", "dv") else e_ds)) - 1 + e_sum) * size[name] +
               store * want[name].abs() for name in size}
        pairs = self.batch * self.p.shape[1] * n  # terms of a bias row, at most
        out["dbias"] = (e_ds + (pairs + 16) * E32) * self.rows(dsa)
        return out

    def dbias_deviation(self):
        """Standard deviation of dBias where delta = dO . O takes O as stored, O in turn from bf16 P: independent
        roundings, each uniform over at most HALF of its value either way, so of variance HALF^2 / 3 of its square.
        A bias row takes each query's delta once, times the pair's P."""
        var = (self.dO.square() * ((((self.p * self.w) @ self.V).square()) + (self.p * self.w).square() @ self.V.square()))
        return self.rows(self.p.square() * var.sum(-1, keepdim=True) * (HALF * HALF / 3)).sqrt()


def over(got, want, bound):
    """How far |got - want| passes the bound at most (<= 0: nowhere)."""
    assert torch.isfinite(got).all()
    return float(((got - want).abs() - bound).max())
