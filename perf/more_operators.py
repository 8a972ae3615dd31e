"""The two ends of a training step around the window attention, as measurable cases.

Three operators, each with a plain form (elementary torch operations, 32 bits,
one rounding at the end; angles and long sums in 64) and the framework's call:

* heads   what stands between the QKV projection and the attention: the norm of
          every head and rotary positions of q and k, read from the projection's
          packed output; forward ("fwd") or backward ("bwd")
* adamw   one AdamW step over all tensors of a model, states in 32 or 8 bits,
          with or without clipping by the gradients' global norm
* norm    the gradients' global norm alone

heads: per head u = N(x) gamma + beta over the head's hd values (N: none, RMS or
layer), then the pairs (a, b) of its first `rot` values turn: y = A (a cos t - b
sin t, a sin t + b cos t), pair i at (i, i + rot / 2) in the half layout and at
(2 i, 2 i + 1) in the interleaved one, t = position along the pair's axis times
its frequency. Pairs are shared out over the axes in order, pairs // axes each and
one more for the last ones; an axis with n pairs has frequencies base^(-j / n).

adamw: t counts steps, c = min(1, max_norm / |g|), g' = c g,
m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
w = w (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
bf16 weights are the rounded copy of fp32 ones. In 8 bits m and r = sqrt(v) are
e4m3 times an fp32 scale of every 256 values (their largest over 448), rounded
to nearest after the step; an r above 0 is held as 2^-9 at least.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.98, 1e-8, 1e-4, 0.05


# ------------------------------------------------------------------ the cases --
def _heads(name, way, dtype, images, grid, heads, hd, rot, layout, kv=0, norm="none", beta=False, packed=True,
           reach=0, scaling="none", factor=1.0, trained=0):
    """reach: positions are given, below this; 0: they are the grid's coordinates. kv: heads of k and v (0: as q)."""
    case = {"op": "heads", "way": way, "dtype": dtype, "images": images, "dims": len(grid), "heads": heads,
            "kv": kv or heads, "hd": hd, "rot": rot, "layout": layout, "norm": norm, "beta": beta, "packed": packed,
            "reach": reach, "scaling": scaling, "factor": factor, "trained": trained}
    case.update({"g%d" % a: g for a, g in enumerate(grid)})
    return dict(case, name=name) if name else case


def _model(name, op, dtype, channels, blocks, bits=32, clip=0.0, grads=""):
    """A stack of blocks. bf16: matrices are bf16 beside fp32 ones, vectors fp32. grads: the type of the matrices'
    gradients (as the matrices where empty)."""
    case = {"op": op, "dtype": dtype, "channels": channels, "blocks": blocks, "grads": grads or dtype}
    if op == "adamw":
        case.update(bits=bits, clip=clip)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one new token of each of eight requests, far along a long context: latency
        _heads("heads_tokens", "fwd", "bf16", 8, (1,), 16, 128, 128, "half", kv=4, norm="rms", packed=False,
               reach=1000000, scaling="yarn", factor=32.0, trained=32768),
        # the 1-degree stage: positions of latitude and longitude in the heads as projected
        _heads("heads_grid1deg_fwd", "fwd", "bf16", 2, (180, 360), 8, 32, 32, "interleaved"),
        # the depth-level stage, positions along all three axes, heads normed; and its gradient
        _heads("heads_depth3d_fwd", "fwd", "bf16", 1, (16, 192, 384), 8, 32, 32, "half", norm="rms"),
        _heads("heads_depth3d_bwd", "bwd", "bf16", 1, (16, 192, 384), 8, 32, 32, "half", norm="rms"),
        # the ragged stage in fp32, half of each head with positions, the gradient
        _heads("heads_ragged_f32_bwd", "bwd", "f32", 1, (181, 362), 12, 32, 16, "interleaved", norm="layer", beta=True),
        # eight heads of 128 on the eddy grid, trained on a coarser one: the gradient, q and k apart
        _heads("heads_wide_bwd", "bwd", "bf16", 1, (256, 540), 8, 128, 128, "half", packed=False, scaling="linear",
               factor=4.0),
        # a step on the smallest grid's model: latency
        _model("adamw_tiny_f32", "adamw", "f32", 32, 1, 32, 1.0),
        # the ragged stage's blocks, mixed precision, clipped
        _model("adamw_stage", "adamw", "bf16", 384, 12, 32, 1.0),
        # the eddy stage's blocks with states in 8 bits
        _model("adamw8_stage", "adamw", "bf16", 512, 12, 8),
        # a large model, its gradients summed in fp32, states in 8 bits, clipped
        _model("adamw8_large", "adamw", "bf16", 1280, 16, 8, 1.0, "f32"),
        # the norm alone: of the 1-degree stage's blocks, and of the large model's gradients
        _model("norm_stage", "norm", "bf16", 256, 6),
        _model("norm_large_f32", "norm", "f32", 1280, 16),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["heads", "heads", "heads", "adamw", "adamw", "norm"])
    if op != "heads":
        while True:
            channels, blocks = 8 * spread(2, 160), spread(1, 32)
            if 12 * channels * channels * blocks <= 200e6:
                break
        dtype = rng.choice(["bf16", "bf16", "f32"])
        grads = rng.choice([dtype, "f32"])
        return _model("", op, dtype, channels, blocks, rng.choice([32, 8]), rng.choice([0.0, 0.5, 1.0]), grads)
    way, dtype = rng.choice(["fwd", "bwd"]), rng.choice(["bf16", "bf16", "f32"])
    hd = rng.choice([16, 32, 32, 64, 80, 96, 128, 128, 256])
    packed = rng.random() < 0.6
    while True:
        kv = spread(1, 32)
        heads = kv if packed else kv * rng.choice([1, 1, 2, 4])
        images, dims = rng.randint(1, 4), rng.choice([1, 2, 2, 3])
        grid = [spread(1, 100000)] if dims == 1 else [spread(1, 24)] * (dims - 2) + [spread(2, 400), spread(2, 600)]
        if images * math.prod(grid) * (heads + 2 * kv) * hd <= 400e6:
            break
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    return _heads("", way, dtype, images, grid, heads, hd, 16 * rng.randint(1, hd // 16), rng.choice(["half", "interleaved"]),
                  kv, rng.choice(["none", "rms", "rms", "layer"]), rng.random() < 0.3, packed,
                  spread(1000, 1000000) if dims == 1 else 0, scaling, 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]),
                  8192 if scaling == "yarn" else 0)


def _grid(case):
    return tuple(case["g%d" % a] for a in range(case["dims"]))


def _sizes(case):
    """Elements of a model's matrices and vectors: the embedding of 69 fields, `blocks` blocks, the head."""
    c, heads = case["channels"], max(1, case["channels"] // 32)
    mats, vecs = [c * 69], [c]
    for _ in range(case["blocks"]):
        mats += [3 * c * c, c * c, 4 * c * c, 4 * c * c]
        vecs += [3 * c, c, 4 * c, c] + [c] * 6 + [15 * 15 * heads]  # projections' biases, two norms and layer scales, positions
    return mats + [69 * 16 * c], vecs + [69 * 16]


def work(case):
    if case["op"] == "heads":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["images"] * math.prod(_grid(case))
        qk, v = rows * (case["heads"] + case["kv"]) * case["hd"], rows * case["kv"] * case["hd"] if case["packed"] else 0
        tensors = 3 if case["way"] == "bwd" and case["norm"] != "none" else 2
        at = 8 * rows if case["reach"] else 0
        return {"bytes": (tensors * qk + 2 * v) * e + at, "flops": (12 if case["way"] == "fwd" else 24) * qk}
    mats, vecs = (sum(s) for s in _sizes(case))
    g = 2 if case["grads"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": g * mats + 4 * vecs, "flops": 2 * (mats + vecs)}
    state = 16 if case["bits"] == 32 else 4 + 16 / 256
    weight = 8 + (2 if case["dtype"] == "bf16" else 0)
    return {"bytes": (g + weight + state) * mats + (4 + 8 + state) * vecs, "flops": 16 * (mats + vecs)}


# ----------------------------------------------------------------- the inputs --
def _frequencies(case):
    """(frequency and axis of every pair, amplitude)."""
    pairs, axes, s = case["rot"] // 2, case["dims"], case["factor"]
    freq, axis = [], []
    for a in range(axes):
        n = pairs // axes + (1 if a >= axes - pairs % axes else 0)
        base = 10000.0 * (s ** (n / (n - 1)) if case["scaling"] == "ntk" and n > 1 else 1.0)
        f = [base ** (-j / n) for j in range(n)]
        if case["scaling"] == "linear":
            f = [x / s for x in f]
        elif case["scaling"] == "yarn":  # turns within the trained length decide: above 32 as they were, below 1 stretched
            ramp = [min(1.0, max(0.0, (case["trained"] * x / (2 * math.pi) - 1) / 31)) for x in f]
            f = [x * ((1 - r) / s + r) for x, r in zip(f, ramp)]
        freq, axis = freq + f, axis + [a] * n
    return freq, axis, 0.1 * math.log(s) + 1 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std + mean).to(dtype)

    st = {"case": dict(case)}
    if case["op"] == "heads":
        dt, grid = DTYPES[case["dtype"]], _grid(case)
        lead, cq, ck = (case["images"],) + grid, case["heads"] * case["hd"], case["kv"] * case["hd"]
        if case["packed"]:  # as the projection leaves it: the heads differ in size
            st["qkv"] = normal(lead + (cq + 2 * ck,), 1.5, 0.2, dt)
            st["q"], st["k"], st["v"] = st["qkv"].split([cq, ck, ck], -1)
        else:
            st["q"], st["k"], st["v"] = normal(lead + (cq,), 1.5, 0.2, dt), normal(lead + (ck,), 1.5, 0.2, dt), None
        for side in "qk":
            some = case["norm"] != "none"
            st[side + "_gamma"] = normal((case["hd"],), 0.2, 1.0) if some else None
            st[side + "_beta"] = normal((case["hd"],), 0.1) if some and case["beta"] else None
        if case["way"] == "bwd":
            st["dq"], st["dk"] = normal(st["q"].shape, dtype=dt), normal(st["k"].shape, dtype=dt)
            st["dv"] = normal(st["v"].shape, dtype=dt) if case["packed"] else None
        freq, axis, amplitude = _frequencies(case)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        st["axis"], st["amplitude"] = torch.tensor(axis, device=dev), amplitude
        st["positions"] = None
        if case["reach"]:
            start = torch.randint(0, case["reach"], (case["images"], 1), generator=gen, device=dev)
            st["positions"] = start + torch.arange(grid[0], device=dev)
        if own:
            from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
            rotary = Rotary(case["rot"], axes=case["dims"], layout=case["layout"], base=10000.0,
                            scaling=None if case["scaling"] == "none" else case["scaling"], factor=case["factor"],
                            trained=case["trained"] or None)
            st["heads"] = AttentionHeads(case["heads"], case["hd"], rotary, norm=case["norm"], eps=1e-5,
                                         dtype=case["dtype"], kv_heads=case["kv"])
        return st
    # tensors of one kind lie in one buffer, each from a multiple of 256 elements on, zeros between them
    for kind, sizes in zip(("mat", "vec"), _sizes(case)):
        first, at = [], 0
        for n in sizes:
            first.append(at)
            at += -(-n // 256) * 256
        here = torch.zeros(at, dtype=torch.bool, device=dev)
        for o, n in zip(first, sizes):
            here[o:o + n] = True
        st[kind + "_at"] = list(zip(first, sizes))
        st[kind + "_grad"] = (normal((at,), 0.002) * here).to(DTYPES[case["grads"]] if kind == "mat" else torch.float32)
        if case["op"] == "adamw":
            w = normal((at,), 0.02 if kind == "mat" else 0.2, 0.0 if kind == "mat" else 0.5) * here
            st[kind + "_master"] = w if kind == "mat" and case["dtype"] == "bf16" else None
            st[kind] = w.to(DTYPES[case["dtype"]]) if kind == "mat" else w
            m, v = normal((at,), 0.001) * here, (0.002 * normal((at,), 0.3, 1.0)) ** 2 * here
            if case["bits"] == 8:
                st[kind + "_m"], st[kind + "_ms"] = _quantised(m)
                st[kind + "_v"], st[kind + "_vs"] = _quantised(torch.sqrt(v))
            else:
                st[kind + "_m"], st[kind + "_v"] = m, v
    st["grads"] = [st[kind + "_grad"][o:o + n] for kind in ("mat", "vec") for o, n in st[kind + "_at"]]
    st["t"] = 100 + seed % 1000
    if own and case["op"] == "adamw":
        from shifted_window_attention_cyclic_gb300.optim import AdamW
        mats, vecs = ([st[kind][o:o + n] for o, n in st[kind + "_at"]] for kind in ("mat", "vec"))
        opt = AdamW([{"params": mats, "weight_decay": DECAY}, {"params": vecs, "weight_decay": 0.0}], lr=LR,
                    betas=(BETA1, BETA2), eps=EPS, state_bits=case["bits"], max_norm=case["clip"] or None)
        opt.steps.fill_(st["t"])
        if st["mat_master"] is not None:
            opt.master.copy_(st["mat_master"])
        opt.m.copy_(torch.cat([st["mat_m"].float(), st["vec_m"].float()]))
        opt.v.copy_(torch.cat([st["mat_v"].float(), st["vec_v"].float()]))
        if case["bits"] == 8:
            opt.m_scale.copy_(torch.cat([st["mat_ms"], st["vec_ms"]]))
            opt.v_scale.copy_(torch.cat([st["mat_vs"], st["vec_vs"]]))
        st["opt"] = opt
    return st


# ------------------------------------------------------------ the plain forms --
def _turns(st):
    """Cosines and sines, times the amplitude, of every token's pairs: [images or 1, tokens, 1, pairs]."""
    case = st["case"]
    if st["positions"] is not None:
        angles = st["positions"].double()[..., None] * st["freq"]
    else:
        grid = _grid(case)
        at = torch.stack(torch.meshgrid(*[torch.arange(g, device=st["q"].device) for g in grid], indexing="ij"), -1)
        angles = (at.view(1, -1, len(grid))[..., st["axis"]].double() * st["freq"])
    angles = angles[:, :, None]
    return torch.cos(angles).float() * st["amplitude"], torch.sin(angles).float() * st["amplitude"]


def _rotated(x, cos, sin, case):
    rot, half = case["rot"], case["rot"] // 2
    if case["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _hat(x, kind):
    mean = x.mean(-1, keepdim=True) if kind == "layer" else 0.0
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5)
    return (x - mean) * rstd, rstd


def _plain_heads(st):
    case = st["case"]
    cos, sin = _turns(st)

    def split(x):
        return x.float().reshape(case["images"], -1, x.shape[-1] // case["hd"], case["hd"])

    def forward(x, gamma, beta):
        u = split(x)
        if case["norm"] != "none":
            u = _hat(u, case["norm"])[0] * gamma
            u = u if beta is None else u + beta
        return _rotated(u, cos, sin, case).to(x.dtype).view(x.shape)

    def backward(x, dy, gamma, beta):
        du = _rotated(split(dy), cos, -sin, case)
        if case["norm"] == "none":
            return du.to(x.dtype).view(x.shape), None, None
        hat, rstd = _hat(split(x), case["norm"])
        g = du * gamma
        mean = g.mean(-1, keepdim=True) if case["norm"] == "layer" else 0.0
        dx = rstd * (g - mean - hat * (g * hat).mean(-1, keepdim=True))
        dgamma = (du * hat).sum((0, 1, 2), dtype=torch.float64).float()
        dbeta = None if beta is None else du.sum((0, 1, 2), dtype=torch.float64).float()
        return dx.to(x.dtype).view(x.shape), dgamma, dbeta

    if case["way"] == "fwd":
        out = {s: forward(st[s], st[s + "_gamma"], st[s + "_beta"]) for s in "qk"}
        if case["packed"]:
            out["v"] = st["v"].clone(memory_format=torch.contiguous_format)
        return out
    out = {}
    for s in "qk":
        out["d" + s], out["d%s_gamma" % s], out["d%s_beta" % s] = backward(st[s], st["d" + s], st[s + "_gamma"], st[s + "_beta"])
    if case["packed"]:
        out["dqkv"] = torch.cat([out.pop("dq"), out.pop("dk"), st["dv"]], -1)
    return out


def _quantised(x):
    """e4m3 values and the scale of every 256."""
    x = x.view(-1, 256)
    top = x.abs().amax(1)
    some = top >= 2.0**-100
    inverse = torch.where(some, 448.0 / top, 0.0)
    q = (x * inverse[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(-1), torch.where(some, top / 448.0, 0.0)


def _held(q, scale):
    return (q.float().view(-1, 256) * scale[:, None]).view(-1)


def _plain_norm(st):
    squares = [st[kind + "_grad"].float().square().sum(dtype=torch.float64) for kind in ("mat", "vec")]
    return torch.sqrt(squares[0] + squares[1]).float()


def _plain_adamw(st):
    case, out = st["case"], {}
    st["t"] += 1
    c = 1.0
    if case["clip"]:
        out["norm"] = _plain_norm(st)
        c = (case["clip"] / out["norm"]).clamp(max=1.0)
    fix1, fix2 = 1.0 - BETA1 ** st["t"], math.sqrt(1.0 - BETA2 ** st["t"])

    def update(kind, decay):
        g = st[kind + "_grad"].float() * c
        if case["bits"] == 8:
            m, v = _held(st[kind + "_m"], st[kind + "_ms"]), _held(st[kind + "_v"], st[kind + "_vs"]).square()
        else:
            m, v = st[kind + "_m"], st[kind + "_v"]
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + g * g * (1.0 - BETA2)
        root = torch.sqrt(v)
        w = st[kind] if st[kind + "_master"] is None else st[kind + "_master"]
        w = w * (1.0 - LR * decay) - (LR / fix1) * m / (root / fix2 + EPS)
        if st[kind + "_master"] is not None:
            st[kind + "_master"].copy_(w)
        st[kind].copy_(w)
        if case["bits"] == 8:
            q, scale = _quantised(m)
            st[kind + "_m"].copy_(q)
            st[kind + "_ms"].copy_(scale)
            q, scale = _quantised(root)
            q = torch.where((root > 0) & (q.float() < 2.0**-9), 2.0**-9, q.float()).to(q.dtype)
            st[kind + "_v"].copy_(q)
            st[kind + "_vs"].copy_(scale)
        else:
            st[kind + "_m"].copy_(m)
            st[kind + "_v"].copy_(v)

    update("mat", DECAY)
    update("vec", 0.0)
    for kind in ("mat", "vec"):
        for name in ("", "_master", "_m", "_v", "_ms", "_vs"):
            if st.get(kind + name) is not None:
                out[kind + name] = st[kind + name]
    return out


# ------------------------------------------------------ the framework's calls --
def _own(st):
    case = st["case"]
    if case["op"] == "heads":
        params = {k: st[k] for k in ("q_gamma", "q_beta", "k_gamma", "k_beta", "positions")}
        if case["way"] == "fwd":
            q, k, v = st["heads"].forward(st["q"], st["k"], st["v"], **params)
            return {"q": q, "k": k, "v": v}
        some = case["norm"] != "none"  # the gradient needs q and k for their norms alone
        g = st["heads"].backward(st["dq"], st["dk"], st["dv"], st["q"] if some else None, st["k"] if some else None,
                                 packed=case["packed"], **params)
        out = g._asdict()
        if case["packed"]:  # one tensor holds the three
            del out["dq"], out["dk"]
        del out["dv"]
        return out
    if case["op"] == "norm":
        from shifted_window_attention_cyclic_gb300.optim import grad_norm
        return {"norm": grad_norm(st["grads"])}
    opt = st["opt"]
    opt.step(st["grads"])
    n = st["mat"].numel()
    out = {"mat": st["mat"], "vec": st["vec"], "mat_master": opt.master, "mat_m": opt.m[:n], "vec_m": opt.m[n:],
           "mat_v": opt.v[:n], "vec_v": opt.v[n:], "norm": opt.grad_norm if case["clip"] else None}
    if case["bits"] == 8:
        out.update(mat_ms=opt.m_scale[:n // 256], vec_ms=opt.m_scale[n // 256:], mat_vs=opt.v_scale[:n // 256],
                   vec_vs=opt.v_scale[n // 256:])
    return out


def run(state):
    if own:
        out = _own(state)
    elif state["case"]["op"] == "heads":
        out = _plain_heads(state)
    else:
        out = {"norm": _plain_norm(state)} if state["case"]["op"] == "norm" else _plain_adamw(state)
    return {k: v for k, v in out.items() if v is not None}


# ------------------------------------------------------------ 64-bit answers --
def exact(case, seed):
    """The definition in float64: rotations as complex products, gradients by autograd."""
    st = prepare(case, seed)
    dev = torch.device("cuda")
    if case["op"] != "heads":
        g = {kind: st[kind + "_grad"].double() for kind in ("mat", "vec")}
        size = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(x) for x in g.values()]))
        if case["op"] == "norm":
            return {"norm": size}
        out, t = {}, st["t"] + 1
        if case["clip"]:
            out["norm"] = size
            g = {kind: x * min(1.0, case["clip"] / float(size)) for kind, x in g.items()}
        for kind, decay in (("mat", DECAY), ("vec", 0.0)):
            m, v = st[kind + "_m"].double(), st[kind + "_v"].double()
            if case["bits"] == 8:
                m = m * st[kind + "_ms"].double().repeat_interleave(256)
                v = (v * st[kind + "_vs"].double().repeat_interleave(256)) ** 2
            m = torch.lerp(g[kind], m, BETA1)
            v = torch.lerp(g[kind] ** 2, v, BETA2)
            w = (st[kind] if st[kind + "_master"] is None else st[kind + "_master"]).double()
            w = w - LR * decay * w - LR * (m / -math.expm1(t * math.log(BETA1))) / ((v / (1 - BETA2**t)).sqrt() + EPS)
            out[kind] = w
            out[kind + "_master"] = w if st[kind + "_master"] is not None else None
            if case["bits"] == 32:
                out.update({kind + "_m": m, kind + "_v": v})
                continue
            for short, x, least in (("m", m, 0.0), ("v", v.sqrt(), 2.0**-9)):
                scale = x.abs().view(-1, 256).amax(1) / 448
                x = torch.nan_to_num(x / scale.repeat_interleave(256))
                q = x.to(torch.float8_e4m3fn).double()
                out[kind + "_" + short] = torch.where(x > 0, q.clamp(min=least), q) if least else q
                out[kind + "_" + short + "s"] = scale
        return out

    freq, axis, amplitude = _frequencies(case)
    grid = _grid(case)
    turn = []
    for f, a in zip(freq, axis):
        if case["reach"]:
            p = st["positions"].double()
        else:
            p = torch.arange(grid[a], dtype=torch.float64, device=dev).view([-1 if b == a else 1 for b in range(len(grid))])
            p = p.expand(grid).reshape(1, -1)
        turn.append(torch.polar(torch.full_like(p, amplitude), p * f))
    turn = torch.stack(turn, -1)[:, :, None]
    rot = case["rot"]

    def forward(x, gamma, beta):
        u = x.unflatten(-1, (-1, case["hd"])).flatten(1, -3)
        if case["norm"] == "layer":
            u = torch.nn.functional.layer_norm(u, u.shape[-1:], gamma, beta, 1e-5)
        elif case["norm"] == "rms":
            u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-5) * gamma
            u = u if beta is None else u + beta
        pairs = u[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else u[..., :rot].unflatten(-1, (-1, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        return torch.cat([z, u[..., rot:]], -1).reshape(x.shape)

    out = {}
    for s in "qk":
        ins = [st[s].double()] + [None if st[s + p] is None else st[s + p].double() for p in ("_gamma", "_beta")]
        if case["way"] == "fwd":
            out[s] = forward(*ins)
            continue
        names = ["d" + s, "d%s_gamma" % s, "d%s_beta" % s]
        some = [i for i in range(3) if ins[i] is not None]
        for i in some:
            ins[i] = ins[i].clone().requires_grad_(True)
        grads = torch.autograd.grad(forward(*ins), [ins[i] for i in some], st["d" + s].double())
        out.update({names[i]: g for i, g in zip(some, grads)})
    if case["packed"]:
        if case["way"] == "fwd":
            out["v"] = st["v"].double()
        else:
            out["dqkv"] = torch.cat([out.pop("dq"), out.pop("dk"), st["dv"].double()], -1)
    return out
