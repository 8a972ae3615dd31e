"""The operators around the window attention that training needs, as measurable cases.

Four operators, each with a plain form (elementary torch operations, 32 bits,
one rounding at the end) and the framework's call:

* attn     shifted-window attention with dropout on its probabilities
* dropout  dropout of activations; `span` consecutive elements share a decision
* norm     the norm before a block, forward ("fwd") or backward ("bwd")
* join     y = x + scale * gate * path * D(N_post(z)), h = N_pre(y); forward or backward

Dropout decisions come from Philox4x32-7 (Salmon et al., "Parallel random
numbers: as easy as 1, 2, 3", 2011) keyed by a 64-bit seed, with counter
(block low, block high, site, step). A block's 128 bits are eight 16-bit
numbers; decision i is number i % 8 of block i // 8 (word (i % 8) // 2, low half
first) and keeps when the number is at least T = round(rate * 65536). Kept
values are scaled by 1 / (1 - T / 65536).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases --
def _attn(name, dtype, batch, grid, window, shift, periodic, heads, hd, land, rate, train):
    lead = (1,) * (3 - len(grid))
    g, w = lead + tuple(grid), lead + tuple(window)
    s, p = (0,) * len(lead) + tuple(shift), (0,) * len(lead) + tuple(periodic)
    case = {"op": "attn", "dtype": dtype, "batch": batch, "dims": len(grid), "heads": heads, "hd": hd, "land": land,
            "rate": rate, "train": train}
    for a in range(3):
        case.update({"g%d" % a: g[a], "w%d" % a: w[a], "s%d" % a: s[a], "p%d" % a: p[a]})
    return dict(case, name=name) if name else case


def _rows(name, op, way, dtype, images, tokens, channels, **more):
    case = dict({"op": op, "way": way, "dtype": dtype, "images": images, "tokens": tokens, "channels": channels}, **more)
    return dict(case, name=name) if name else case


def listed():
    return [
        # a fine-tuning step on the smallest fp32 grid: latency
        _attn("attn_tiny_f32_train", "f32", 1, (16, 32), (4, 8), (2, 4), (0, 0), 2, 16, 0.0, 0.1, True),
        # the 1-degree stage, dropout kept on at inference for an ensemble: forward alone
        _attn("attn_grid1deg_fwd", "bf16", 2, (180, 360), (6, 12), (3, 6), (0, 1), 8, 32, 0.0, 0.1, False),
        # ragged windows at every edge, a training step
        _attn("attn_ragged_train", "bf16", 1, (181, 362), (8, 8), (4, 4), (0, 1), 12, 32, 0.0, 0.1, True),
        # the eddy-resolving ocean stage with its land mask, a training step
        _attn("attn_eddy_train", "bf16", 1, (256, 540), (8, 12), (4, 6), (0, 1), 16, 32, 0.3, 0.2, True),
        # the norm that opens a block of the depth-level stage
        _rows("norm_depth3d_fwd", "norm", "fwd", "bf16", 1, 16 * 192 * 384, 256, kind="layer", affine=True),
        # its gradient on the ragged stage in fp32, with the residual's gradient added
        _rows("norm_ragged_f32_bwd", "norm", "bwd", "f32", 1, 181 * 362, 384, kind="rms", affine=True),
        # the join after the attention of the smallest grid: latency
        _rows("join_tiny_fwd", "join", "fwd", "bf16", 1, 16 * 32, 64, post="none", pre="layer", scale=True, gate=False,
              rate=0.0, path=0.0),
        # the eddy stage with a norm on both sides, a gate per image, dropout
        _rows("join_eddy_fwd", "join", "fwd", "bf16", 1, 256 * 540, 512, post="rms", pre="layer", scale=True, gate=True,
              rate=0.1, path=0.0),
        # the 1-degree stage backward: per-image gates, stochastic depth
        _rows("join_grid1deg_bwd", "join", "bwd", "bf16", 2, 180 * 360, 256, post="layer", pre="layer", scale=True,
              gate=True, rate=0.1, path=0.2),
        # a stage of 8 heads of 128 channels on an odd grid, backward
        _rows("join_wide_bwd", "join", "bwd", "bf16", 3, 181 * 91, 1024, post="rms", pre="rms", scale=True, gate=False,
              rate=0.0, path=0.0),
        # dropout after the embedding of one small image, and stochastic depth over the depth-level stage's activations
        _rows("dropout_tiny_f32", "dropout", "fwd", "f32", 1, 16 * 32, 32, span=1, rate=0.1),
        _rows("dropout_depth3d", "dropout", "fwd", "bf16", 1, 16 * 192 * 384, 256, span=1, rate=0.1),
    ]


def draw(rng):
    op = rng.choice(["attn", "attn", "norm", "norm", "join", "join", "join", "dropout"])

    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if op == "attn":
        f32 = rng.random() < 0.25
        dims = rng.choice([2, 2, 3])
        while True:
            window = [rng.randint(1, 4)] * (dims - 2) + [rng.randint(2, 12), rng.randint(2, 16)]
            grid = [spread(max(2, w), 24) for w in window[:dims - 2]] + [spread(12, 200), spread(12, 400)]
            heads, hd, batch = rng.randint(1, 16), rng.choice([16, 32]) if f32 else 32, rng.randint(1, 2)
            slots, tokens = math.prod(window), math.prod(grid)
            most = 2e6 if f32 else 256 * 540 * 16 * 96
            if slots <= 128 and batch * tokens * heads * max(slots, 32) <= most:
                break
        shift = [rng.choice([0, w // 2 if g > w // 2 else 0]) for w, g in zip(window, grid)]
        return _attn("", "f32" if f32 else "bf16", batch, grid, window, shift, [rng.randint(0, 1) for _ in grid], heads, hd,
                     rng.choice([0.0, 0.3]), rng.choice([0.05, 0.1, 0.2, 0.5]), rng.random() < 0.6)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        channels, images, tokens = 8 * spread(2, 512), rng.randint(1, 4), spread(64, 1200000)
        if images * tokens * channels <= 140e6:
            break
    if op == "dropout":
        return _rows("", op, "fwd", dtype, images, tokens, channels, span=rng.choice([1, 1, channels, tokens * channels]),
                     rate=rng.choice([0.05, 0.1, 0.3, 0.5]))
    way = rng.choice(["fwd", "bwd"])
    if op == "norm":
        return _rows("", op, way, dtype, images, tokens, channels, kind=rng.choice(["layer", "rms"]), affine=rng.random() < 0.8)
    return _rows("", op, way, dtype, images, tokens, channels, post=rng.choice(["none", "layer", "rms"]),
                 pre=rng.choice(["none", "layer", "rms"]), scale=rng.random() < 0.7, gate=rng.random() < 0.5,
                 rate=rng.choice([0.0, 0.1, 0.3]), path=rng.choice([0.0, 0.2]))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attn":
        tokens = case["batch"] * case["g0"] * case["g1"] * case["g2"]
        slots = case["w0"] * case["w1"] * case["w2"]
        c = case["heads"] * case["hd"]
        small = 4 * tokens * case["heads"] + (tokens if case["land"] else 0)
        if case["train"]:
            return {"bytes": 8 * tokens * c * e + small, "flops": 14 * tokens * slots * c}
        return {"bytes": 4 * tokens * c * e + small, "flops": 4 * tokens * slots * c}
    n = case["images"] * case["tokens"] * case["channels"]
    if case["op"] == "dropout":
        return {"bytes": 2 * n * e, "flops": 2 * n}
    if case["op"] == "norm":
        return {"bytes": (2 if case["way"] == "fwd" else 4) * n * e, "flops": (8 if case["way"] == "fwd" else 16) * n}
    pre = 1 if case["pre"] != "none" else 0
    if case["way"] == "fwd":
        return {"bytes": (3 + pre) * n * e, "flops": 20 * n}
    # without a post norm, scale and gate, the gradient of z needs no z
    needs_z = case["post"] != "none" or case["scale"] or case["gate"]
    needs_y = pre == 1
    return {"bytes": (3 + pre + needs_z + needs_y) * n * e, "flops": 40 * n}


# ----------------------------------------------------------------- the inputs --
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std + mean).to(dtype)

    st = {"case": dict(case), "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % 2**64, "step": seed % 1000 + 1}
    if case["op"] == "attn":
        grid = tuple(case["g%d" % a] for a in range(3 - case["dims"], 3))
        window, shift, periodic = (tuple(case[k + "%d" % a] for a in range(3 - case["dims"], 3)) for k in "wsp")
        shape = (case["batch"],) + grid + (case["heads"] * case["hd"],)
        for name in ("q", "k", "v", "dout"):
            st[name] = normal(shape, dtype=dt)
        rows = math.prod(2 * w - 1 for w in window)
        st["bias"] = normal((rows, case["heads"]), 0.02)
        st["land"] = None
        if case["land"]:
            # land comes in patches of 8 x 8 tokens, the same at every depth
            lat, lon = grid[-2], grid[-1]
            xi = torch.rand((case["batch"], -(-lat // 8), -(-lon // 8)), generator=gen, device=dev) < case["land"]
            xi = xi.repeat_interleave(8, 1).repeat_interleave(8, 2)[:, :lat, :lon].to(torch.uint8)
            if len(grid) == 3:
                xi = xi[:, None].expand(-1, grid[0], -1, -1)
            st["land"] = xi.contiguous()
        st.update(_tables(grid, window, shift, periodic, dev))
        if own:
            from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
            from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
            st["attn"] = SwinWindowAttention(grid, window, shift, periodic, case["heads"], case["hd"], case["batch"],
                                             case["dtype"], bool(case["land"]))
            st["drop"] = Dropout(DropoutState(st["seed"], st["step"]), case["rate"], site=7)
        return st
    b, t, c = case["images"], case["tokens"], case["channels"]
    shape = (b, t, c)
    if case["op"] == "dropout":
        st["x"] = normal(shape, dtype=dt)
    elif case["op"] == "norm":
        st["x"] = normal(shape, 1.5, 0.3, dt)
        st["gamma"] = normal((c,), 0.2, 1.0) if case["affine"] else None
        st["beta"] = normal((c,), 0.1) if case["affine"] else None
        if case["way"] == "bwd":
            st["dh"] = normal(shape, dtype=dt)
            st["dres"] = normal(shape, dtype=dt)
    else:
        st["x"] = normal(shape, 1.5, 0.3, dt)  # the residual stream: x forward, y (as stored) backward
        st["z"] = normal(shape, 0.8, 0.1, dt)
        for side in ("post", "pre"):
            some = case[side] != "none"
            st[side + "_gamma"] = normal((c,), 0.2, 1.0) if some else None
            st[side + "_beta"] = normal((c,), 0.1) if case[side] == "layer" else None
        st["scale"] = normal((c,), 0.05, 0.3) if case["scale"] else None
        st["gate"] = normal((b, c), 0.3, 0.8) if case["gate"] else None
        if case["way"] == "bwd":
            st["dy"] = normal(shape, dtype=dt)
            st["dh"] = normal(shape, dtype=dt) if case["pre"] != "none" else None
    if own:
        from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
        from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
        rng = DropoutState(st["seed"], st["step"])
        st["drop"] = Dropout(rng, case["rate"], site=7) if case.get("rate") else None
        st["path"] = Dropout(rng, case["path"], site=8) if case.get("path") else None
        if case["op"] == "norm":
            st["norm"] = BlockNorm(c, case["kind"], 1e-5, case["dtype"])
        elif case["op"] == "join":
            st["join"] = ResidualJoin(c, case["post"], case["pre"], 1e-5, case["dtype"])
    return st


def _tables(grid, window, shift, periodic, dev):
    """The routing that a plan keeps: token of every window slot (-1 = pad), its region code, bias row of a slot pair."""
    lead = (1,) * (3 - len(grid))
    g, w = lead + grid, lead + window
    s, p = (0,) * len(lead) + shift, (0,) * len(lead) + periodic
    win = [-(-g[a] // w[a]) for a in range(3)]

    def along(a):
        """Window coordinate and slot coordinate of dim a, over [nwin] and [n]."""
        shape_w, shape_s = [1, 1, 1], [1, 1, 1]
        shape_w[a], shape_s[a] = win[a], w[a]
        ww = torch.arange(win[a], device=dev).view(shape_w).expand(win).reshape(-1, 1)
        ss = torch.arange(w[a], device=dev).view(shape_s).expand(w).reshape(1, -1)
        pos = ww * w[a] + ss
        ok = pos < g[a]
        return torch.where(ok, (pos + s[a]) % g[a], 0), ok, (pos >= g[a] - s[a]) & (s[a] > 0) & (not p[a]), ss.reshape(-1)

    u0, ok0, r0, s0 = along(0)
    u1, ok1, r1, s1 = along(1)
    u2, ok2, r2, s2 = along(2)
    src = torch.where(ok0 & ok1 & ok2, (u0 * g[1] + u1) * g[2] + u2, -1)
    region = r0.long() + 2 * r1.long() + 4 * r2.long()
    rel = (s0[:, None] - s0 + w[0] - 1) * (2 * w[1] - 1) + s1[:, None] - s1 + w[1] - 1
    rel = rel * (2 * w[2] - 1) + s2[:, None] - s2 + w[2] - 1
    return {"src": src, "region": region, "rel": rel}


# ------------------------------------------------------------ the plain forms --
def _keep(st, site, blocks, rate):
    """Decisions (bool [..., 8]) of the Philox blocks `blocks` (int64)."""
    seed, m = st["seed"], 0xFFFFFFFF
    c0, c1 = blocks & m, blocks >> 32
    c2, c3 = torch.full_like(blocks, site), torch.full_like(blocks, st["step"])
    k0, k1 = seed & m, seed >> 32
    for _ in range(7):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m) ^ c1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    words = torch.stack([c0, c1, c2, c3], -1)
    halves = torch.stack([words & 0xFFFF, words >> 16], -1).flatten(-2)
    return halves >= round(rate * 65536)


def _kept(rate):
    return 1.0 / (1.0 - round(rate * 65536) / 65536)


def _keep_flat(st, site, n, rate, dev):
    return _keep(st, site, torch.arange(-(-n // 8), device=dev), rate).view(-1)[:n]


def _plain_attn(st):
    case = st["case"]
    b, h, hd, src, region = case["batch"], case["heads"], case["hd"], st["src"], st["region"]
    dt, n, tokens = DTYPES[case["dtype"]], src.shape[1], case["g0"] * case["g1"] * case["g2"]
    at = src.clamp(min=0)

    def windows(x):  # [B, grid, C] -> [B, nwin, H, n, hd]
        return x.view(b, tokens, h, hd)[:, at].permute(0, 1, 3, 2, 4).float()

    def grid(x, like):  # the inverse route
        out = torch.empty((b, tokens, h, hd), dtype=dt, device=x.device)
        out[:, src[src >= 0]] = x.permute(0, 1, 3, 2, 4)[:, src >= 0].to(dt)
        return out.view(like.shape)

    q, k, v = windows(st["q"]), windows(st["k"]), windows(st["v"])
    live = (src >= 0)[None]
    if st["land"] is not None:
        live = live & (st["land"].view(b, tokens)[:, at] == 0)
    visible = (live[:, :, None, :] & live[:, :, :, None] & (region[:, :, None] == region[:, None, :])[None])[:, :, None]
    s = q @ k.transpose(-1, -2) * hd**-0.5 + st["bias"][st["rel"]].permute(2, 0, 1)
    s = s.masked_fill(~visible, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    p = p / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    # decisions of query token t and key slot j: block ((b H + h) N + t) ceil(n / 8) + j / 8
    row = (torch.arange(b * h, device=s.device).view(b, 1, h, 1) * tokens + at[None, :, None, :])[..., None]
    nb = -(-n // 8)
    keep = _keep(st, 7, row * nb + torch.arange(nb, device=s.device), case["rate"]).flatten(-2)[..., :n]
    weight = keep * _kept(case["rate"])
    pd = p * weight
    lse_grid = torch.empty((b, h, tokens), dtype=torch.float32, device=s.device)
    lse_grid[:, :, src[src >= 0]] = lse.permute(0, 2, 1, 3)[:, :, src >= 0]
    out = {"o": grid(pd @ v, st["q"]), "lse": lse_grid.view((b, h) + st["q"].shape[1:-1])}
    if not case["train"]:
        return out
    do = windows(st["dout"])
    dp = do @ v.transpose(-1, -2) * weight
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    out["dq"] = grid(ds @ k * hd**-0.5, st["q"])
    out["dk"] = grid(ds.transpose(-1, -2) @ q * hd**-0.5, st["q"])
    out["dv"] = grid(pd.transpose(-1, -2) @ do, st["q"])
    pairs = ds.sum((0, 1), dtype=torch.float64).flatten(1)
    dbias = torch.zeros((st["bias"].shape[0], h), dtype=torch.float64, device=s.device)
    out["dbias"] = dbias.index_add(0, st["rel"].flatten(), pairs.t()).float()
    return out


def _hat(x, kind):
    """The normalised rows of x and 1 / their deviation."""
    mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5)
    return (x - mean) * rstd, rstd


def _affine(x, gamma, beta):
    x = x if gamma is None else x * gamma
    return x if beta is None else x + beta


def _norm_grad(g, hat, rstd, kind):
    m = g.mean(-1, keepdim=True) if kind == "layer" else 0.0
    return rstd * (g - m - hat * (g * hat).mean(-1, keepdim=True))


def _columns(x):
    return x.sum((0, 1), dtype=torch.float64).float()


def _plain_norm(st):
    case, x = st["case"], st["x"].float()
    hat, rstd = _hat(x, case["kind"])
    if case["way"] == "fwd":
        return {"h": _affine(hat, st["gamma"], st["beta"]).to(st["x"].dtype)}
    dh = st["dh"].float()
    g = dh if st["gamma"] is None else dh * st["gamma"]
    out = {"dx": (st["dres"].float() + _norm_grad(g, hat, rstd, case["kind"])).to(st["x"].dtype)}
    if case["affine"]:
        out.update(dgamma=_columns(dh * hat), dbeta=_columns(dh))
    return out


def _weights(st):
    """What the branch is multiplied by: channel scale and image gate apart from the dropouts."""
    case, x = st["case"], st["x"]
    b, t, c = x.shape
    w = torch.ones((1, 1, 1), device=x.device)
    if st["scale"] is not None:
        w = w * st["scale"]
    if st["gate"] is not None:
        w = w * st["gate"][:, None]
    d = torch.ones((1, 1, 1), device=x.device)
    if case["rate"]:
        d = d * (_keep_flat(st, 7, b * t * c, case["rate"], x.device).view(b, t, c) * _kept(case["rate"]))
    if case["path"]:
        d = d * (_keep_flat(st, 8, b, case["path"], x.device).view(b, 1, 1) * _kept(case["path"]))
    return w, d


def _plain_join(st):
    case, dt = st["case"], st["x"].dtype
    x, z = st["x"].float(), st["z"].float()
    w, d = _weights(st)
    zhat, zr = _hat(z, case["post"]) if case["post"] != "none" else (z, None)
    u = _affine(zhat, st["post_gamma"], st["post_beta"])
    if case["way"] == "fwd":
        y = (x + w * d * u).to(dt)
        out = {"y": y}
        if case["pre"] != "none":
            out["h"] = _affine(_hat(y.float(), case["pre"])[0], st["pre_gamma"], st["pre_beta"]).to(dt)
        return out
    g, out = st["dy"].float(), {}
    if case["pre"] != "none":
        dh = st["dh"].float()
        yhat, yr = _hat(x, case["pre"])
        g = g + _norm_grad(dh * st["pre_gamma"], yhat, yr, case["pre"])
        out["dpre_gamma"] = _columns(dh * yhat)
        if case["pre"] == "layer":
            out["dpre_beta"] = _columns(dh)
    out["dx"] = g.to(dt)
    gd = g * d
    du = gd * w
    if case["post"] != "none":
        out["dpost_gamma"] = _columns(du * zhat)
        if case["post"] == "layer":
            out["dpost_beta"] = _columns(du)
        out["dz"] = _norm_grad(du * st["post_gamma"], zhat, zr, case["post"]).to(dt)
    else:
        out["dz"] = du.expand_as(z).to(dt)
    if st["scale"] is not None:
        out["dscale"] = _columns(gd * u if st["gate"] is None else gd * u * st["gate"][:, None])
    if st["gate"] is not None:
        out["dgate"] = (gd * u if st["scale"] is None else gd * u * st["scale"]).sum(1, dtype=torch.float64).float()
    return out


def _plain_dropout(st):
    case, x = st["case"], st["x"]
    keep = _keep_flat(st, 7, -(-x.numel() // case["span"]), case["rate"], x.device)
    if case["span"] > 1:
        keep = keep.repeat_interleave(case["span"])[:x.numel()]
    return {"y": (x.float() * keep.view(x.shape) * _kept(case["rate"])).to(x.dtype)}


# ------------------------------------------------------ the framework's calls --
def _own(st):
    case = st["case"]
    if case["op"] == "attn":
        attn = st["attn"]
        o, lse = attn.forward(st["q"], st["k"], st["v"], st["bias"], st["land"], dropout=st["drop"])
        if not case["train"]:
            return {"o": o, "lse": lse}
        dq, dk, dv, dbias = attn.backward(st["q"], st["k"], st["v"], st["dout"], lse, st["bias"], st["land"], o=o,
                                          dropout=st["drop"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "dbias": dbias}
    if case["op"] == "dropout":
        from shifted_window_attention_cyclic_gb300.dropout import apply_dropout
        return {"y": apply_dropout(st["x"], st["drop"], span=case["span"])}
    if case["op"] == "norm":
        if case["way"] == "fwd":
            return {"h": st["norm"].forward(st["x"], st["gamma"], st["beta"])}
        dx, dgamma, dbeta = st["norm"].backward(st["x"], st["dh"], st["gamma"], st["beta"], dres=st["dres"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    params = {k: st[k] for k in ("post_gamma", "post_beta", "scale", "gate", "pre_gamma", "pre_beta", "drop", "path")}
    if case["way"] == "fwd":
        y, h = st["join"].forward(st["x"], st["z"], **params)
        return {"y": y, "h": h}
    return st["join"].backward(st["x"], st["z"], st["dy"], st["dh"], **params)._asdict()


def run(state):
    if own:
        out = _own(state)
        return {k: v for k, v in out.items() if v is not None}
    return {"attn": _plain_attn, "dropout": _plain_dropout, "norm": _plain_norm, "join": _plain_join}[state["case"]["op"]](state)


# ------------------------------------------------------------ 64-bit answers --
def exact(case, seed):
    """The definition in float64: whole-tensor autograd, decisions from numpy."""
    st = prepare(case, seed)
    dev = torch.device("cuda")

    def decide(site, first, rate):
        """Weights (0 or 1 / kept share) [len(first), 8] of the Philox blocks in the numpy uint64 array `first`."""
        lo32 = np.uint64(0xFFFFFFFF)
        ctr = [first & lo32, first >> np.uint64(32), np.full_like(first, site), np.full_like(first, st["step"])]
        for r in range(7):
            ka = np.uint64((st["seed"] % 2**32 + r * 0x9E3779B9) % 2**32)
            kb = np.uint64((st["seed"] // 2**32 + r * 0xBB67AE85) % 2**32)
            a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
            ctr = [(b >> np.uint64(32)) ^ ctr[1] ^ ka, b & lo32, (a >> np.uint64(32)) ^ ctr[3] ^ kb, a & lo32]
        u = np.empty((first.size, 8), np.uint16)
        for i in range(4):
            u[:, 2 * i] = (ctr[i] & np.uint64(0xFFFF)).astype(np.uint16)
            u[:, 2 * i + 1] = (ctr[i] >> np.uint64(16)).astype(np.uint16)
        t = int(np.rint(rate * 65536))
        return torch.from_numpy(u.astype(np.int32)).to(dev).ge(t).double() * (65536.0 / (65536 - t))

    def decide_flat(site, n, rate):
        return decide(site, np.arange(-(-n // 8), dtype=np.uint64), rate).reshape(-1)[:n]

    def f64(x):
        return None if x is None else x.double()

    if case["op"] == "dropout":
        w = decide_flat(7, -(-st["x"].numel() // case["span"]), case["rate"])
        if case["span"] > 1:
            w = w[:, None].expand(-1, case["span"]).reshape(-1)
        return {"y": f64(st["x"]) * w[:st["x"].numel()].view(st["x"].shape)}

    def normed(x, kind, gamma, beta):
        if kind == "none":
            return x
        if kind == "layer":
            return torch.nn.functional.layer_norm(x, x.shape[-1:], gamma, beta, 1e-5)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)
        x = x if gamma is None else x * gamma
        return x if beta is None else x + beta

    if case["op"] == "norm":
        x, gamma, beta = f64(st["x"]), f64(st["gamma"]), f64(st["beta"])
        if case["way"] == "fwd":
            return {"h": normed(x, case["kind"], gamma, beta)}
        ins = [x] + ([gamma, beta] if case["affine"] else [])
        for t in ins:
            t.requires_grad_(True)
        grads = torch.autograd.grad(normed(x, case["kind"], gamma, beta), ins, f64(st["dh"]))
        out = {"dx": grads[0] + f64(st["dres"])}
        if case["affine"]:
            out.update(dgamma=grads[1], dbeta=grads[2])
        return out

    if case["op"] == "join":
        x, z = f64(st["x"]), f64(st["z"])
        names = ["post_gamma", "post_beta", "scale", "gate", "pre_gamma", "pre_beta"]
        par = {k: f64(st[k]) for k in names}
        d = torch.ones((1, 1, 1), dtype=torch.float64, device=dev)
        if case["rate"]:
            d = d * decide_flat(7, x.numel(), case["rate"]).view(x.shape)
        if case["path"]:
            d = d * decide_flat(8, x.shape[0], case["path"]).view(-1, 1, 1)
        if case["way"] == "bwd":
            for t in [x, z] + list(par.values()):
                if t is not None:
                    t.requires_grad_(True)
        branch = normed(z, case["post"], par["post_gamma"], par["post_beta"]) * d
        if par["scale"] is not None:
            branch = branch * par["scale"]
        if par["gate"] is not None:
            branch = branch * par["gate"][:, None, :]
        if case["way"] == "fwd":
            y = x + branch
            out = {"y": y}
            if case["pre"] != "none":
                stored = y.to(DTYPES[case["dtype"]]).double()
                out["h"] = normed(stored, case["pre"], par["pre_gamma"], par["pre_beta"])
            return out
        # x holds y as stored: its gradient is dy plus the norm's, and reaches the branch unchanged
        out, g = {}, f64(st["dy"])
        if case["pre"] != "none":
            ins = [x] + [par[k] for k in ("pre_gamma", "pre_beta") if par[k] is not None]
            grads = torch.autograd.grad(normed(x, case["pre"], par["pre_gamma"], par["pre_beta"]), ins, f64(st["dh"]))
            g = g + grads[0]
            out.update(zip(["d" + k for k in ("pre_gamma", "pre_beta") if par[k] is not None], grads[1:]))
        some = [k for k in ("post_gamma", "post_beta", "scale", "gate") if par[k] is not None]
        grads = torch.autograd.grad(branch, [z] + [par[k] for k in some], g)
        out.update(zip(["d" + k for k in some], grads[1:]))
        out.update(dx=g, dz=grads[0])
        return out

    # attention: roll, pad, cut into windows; gradients by autograd
    b, h, hd = case["batch"], case["heads"], case["hd"]
    g, w, s, per = (tuple(case[k + str(a)] for a in range(3)) for k in "gwsp")
    win = tuple(-(-g[a] // w[a]) for a in range(3))
    n, tokens = w[0] * w[1] * w[2], g[0] * g[1] * g[2]

    def cut(x, fill):
        """[B, g0, g1, g2, X] -> [B, nwin, n, X]; pads hold `fill`."""
        x = torch.roll(x, (-s[0], -s[1], -s[2]), (1, 2, 3))
        full = torch.full((x.shape[0],) + tuple(win[a] * w[a] for a in range(3)) + x.shape[4:], fill, dtype=x.dtype, device=dev)
        full[:, :g[0], :g[1], :g[2]] = x
        full = full.view(x.shape[0], win[0], w[0], win[1], w[1], win[2], w[2], -1).permute(0, 1, 3, 5, 2, 4, 6, 7)
        return full.reshape(x.shape[0], win[0] * win[1] * win[2], n, -1)

    def paste(x):
        x = x.view(x.shape[0], win[0], win[1], win[2], w[0], w[1], w[2], -1).permute(0, 1, 4, 2, 5, 3, 6, 7)
        x = x.reshape(x.shape[0], win[0] * w[0], win[1] * w[1], win[2] * w[2], -1)[:, :g[0], :g[1], :g[2]]
        return torch.roll(x, s, (1, 2, 3))

    q, k, v = (f64(st[x]).view(b, *g, h * hd) for x in ("q", "k", "v"))
    bias = f64(st["bias"])
    if case["train"]:
        for t in (q, k, v, bias):
            t.requires_grad_(True)
    heads = [cut(x, 0.0).view(b, -1, n, h, hd).transpose(2, 3) for x in (q, k, v)]
    token = cut(torch.arange(tokens, device=dev).view(1, *g, 1), -1)[0, :, :, 0]
    sea = torch.ones((b, *g, 1), dtype=torch.int64, device=dev) if st["land"] is None else (st["land"] == 0).long().view(b, *g, 1)
    live = cut(sea, 0)[..., 0] == 1
    coord = [torch.arange(g[a], device=dev) for a in range(3)]
    part = [((c - s[a]) % g[a] >= g[a] - s[a]).long() * (1 if s[a] and not per[a] else 0) for a, c in enumerate(coord)]
    label = part[0][:, None, None] * 4 + part[1][None, :, None] * 2 + part[2][None, None, :]
    label = cut(label.view(1, *g, 1), 0)[0, :, :, 0]
    mask = live[:, :, :, None] & live[:, :, None, :] & (label[:, :, None] == label[:, None, :])
    slot = torch.stack(torch.meshgrid(*[torch.arange(x, device=dev) for x in w], indexing="ij")).flatten(1)
    diff = [slot[a][:, None] - slot[a][None, :] + w[a] - 1 for a in range(3)]
    pair = (diff[0] * (2 * w[1] - 1) + diff[1]) * (2 * w[2] - 1) + diff[2]
    logits = heads[0] @ heads[1].transpose(-1, -2) / math.sqrt(hd) + bias[pair].permute(2, 0, 1)
    logits = torch.where(mask[:, :, None], logits, torch.full((), -math.inf, dtype=torch.float64, device=dev))
    lse = torch.logsumexp(logits, -1, keepdim=True)
    prob = torch.exp(logits - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))
    nb = -(-n // 8)
    tok = token.clamp(min=0).cpu().numpy().astype(np.uint64)
    rows = (np.arange(b * h, dtype=np.uint64) * np.uint64(tokens)).reshape(b, 1, h, 1) + tok[None, :, None, :]
    blocks = rows[..., None] * np.uint64(nb) + np.arange(nb, dtype=np.uint64)
    drop = decide(7, blocks.reshape(-1), case["rate"]).view(b, -1, h, n, nb * 8)[..., :n]
    o = paste(((prob * drop) @ heads[2]).transpose(2, 3).reshape(b, -1, n, h * hd)).reshape(st["q"].shape)
    shape = (b, h) + tuple(st["q"].shape[1:-1])
    out = {"o": o.detach(), "lse": paste(lse[..., 0].transpose(2, 3)).permute(0, 4, 1, 2, 3).reshape(shape).detach()}
    if case["train"]:
        grads = torch.autograd.grad(o, [q, k, v, bias], f64(st["dout"]))
        out.update(dq=grads[0].reshape(o.shape), dk=grads[1].reshape(o.shape), dv=grads[2].reshape(o.shape), dbias=grads[3])
    return out
