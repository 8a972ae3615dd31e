"""The norm, the residual join and dropout on the GPU against the 64-bit
references, over widths, row counts, types and which parameters are present.

Tolerances. Every output is a sum of terms computed in fp32; the reference
gives the sum `size` of the terms' absolute values. A row's statistics come
from at most 16 sums in a thread, 5 shuffles and 16 warps, and a value passes
about as many roundings again on the way out: OPS = 96 roundings of
2^-24 each bound the relative error of what a row computes, times 1 + |mean| /
deviation for the cancellation in x - mean; where an output holds xhat itself,
its size counts (|x| + mean |x|) / deviation, because x - mean can be far
smaller than the rounding of the mean. Column sums add up to LONG more
roundings (one per row of a thread, then the fold). Outputs of bf16 add half a
step, 2^-8 of the value."""
import pytest

torch = pytest.importorskip("torch")

from tests import rows_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

OPS = 96 * 2.0**-24
LONG = 256 * 2.0**-24
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return 2.0**-8 if dtype == "bf16" else 2.0**-24


def close(name, got, want, size, fp32, store=2.0**-24):
    """|got - want| <= fp32 * size + store * |want|, elementwise."""
    got, want = got.double().cpu().reshape(want.shape), want
    bound = fp32 * size + store * want.abs() + 1e-30
    bad = (got - want).abs() - bound
    assert torch.isfinite(got).all() and (bad <= 0).all(), "%s: over the bound by %.3e (error %.3e, bound %.3e)" % (
        name, bad.max(), (got - want).abs().max(), bound.max())


def cond(x, kind, eps=1e-5):
    """1 + |mean| / deviation of each row."""
    mean, rstd = ref.stats(x, kind, eps)
    return 1 + mean.abs() * rstd


def make(gen, shape, dtype, std=1.0, mean=0.0):
    t = (torch.randn(shape, generator=gen) * std + mean).to(TDT[dtype])
    return t.cuda(), t.double()


def param(gen, shape, std, mean, present=True):
    if not present:
        return None, None
    t = torch.randn(shape, generator=gen) * std + mean
    return t.cuda(), t.double()


WIDTHS = [8, 24, 32, 40, 64, 72, 96, 128, 136, 184, 200, 256, 264, 384, 392, 512, 520, 768, 1024, 1032, 1536, 2048, 2056,
          2320, 4096, 4104, 5000, 8192]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("channels", WIDTHS)
def test_norm(channels, dtype):
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm
    gen = torch.Generator().manual_seed(channels)
    for k, (b, t) in enumerate([(1, 1), (2, 37), (1, 613)]):
        kind = ("layer", "rms")[(k + channels // 8) % 2]
        x, x64 = make(gen, (b, t, channels), dtype, 1.5, 3.0)
        dh, dh64 = make(gen, (b, t, channels), dtype)
        dres, dres64 = make(gen, (b, t, channels), dtype) if k != 1 else (None, 0.0 * dh64)
        gamma, gamma64 = param(gen, (channels,), 0.3, 1.0, k != 2)
        beta, beta64 = param(gen, (channels,), 0.3, 0.0, k == 0)
        norm = BlockNorm(channels, kind, 1e-5, dtype)
        c = cond(x64, kind)
        want = ref.norm_fwd(x64, kind, 1e-5, gamma64, beta64)
        size = want.abs() if beta is None else want.abs() + 2 * beta64.abs()
        # x - mean is off by the mean's error: OPS |x| rstd |gamma| whatever the difference
        _, rstd = ref.stats(x64, kind, 1e-5)
        size = size + x64.abs().mean(-1, keepdim=True) * rstd * (1.0 if gamma is None else gamma64.abs())
        close("h", norm.forward(x, gamma, beta), want, size, OPS, half_step(dtype))
        dx, dgamma, dbeta = norm.backward(x, dh, gamma, beta, dres)
        w, tg, tb, s = ref.norm_bwd(x64, dh64, kind, 1e-5, gamma64)
        close("dx", dx, w + dres64, c * s + dres64.abs(), OPS, half_step(dtype))
        assert (dgamma is None) == (gamma is None) and (dbeta is None) == (beta is None)
        if gamma is not None:
            close("dgamma", dgamma, tg.sum((0, 1)), (tg.abs() + c * dh64.abs()).sum((0, 1)), OPS + LONG)
        if beta is not None:
            close("dbeta", dbeta, tb.sum((0, 1)), tb.abs().sum((0, 1)), LONG)


JOINS = [("none", "none"), ("none", "layer"), ("layer", "none"), ("rms", "layer"), ("layer", "rms"), ("rms", "rms")]


def join_case(seed, b, t, channels, dtype, post, pre, present, rate, path_rate):
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    gen = torch.Generator().manual_seed(seed)
    case = {n: make(gen, (b, t, channels), dtype, 1.0, 0.3) for n in ("x", "z", "dy", "dh")}
    par, par64 = {}, {}
    for n, shape, std, mean in (("post_gamma", (channels,), 0.3, 1.0), ("post_beta", (channels,), 0.3, 0.0),
                                ("scale", (channels,), 0.1, 0.5), ("gate", (b, channels), 0.5, 0.5),
                                ("pre_gamma", (channels,), 0.3, 1.0), ("pre_beta", (channels,), 0.3, 0.0)):
        some = n in present and not (n.startswith("post") and post == "none") and not (n.startswith("pre") and pre == "none")
        par[n], par64[n] = param(gen, shape, std, mean, some)
    key, step = 0x9E3779B97F4A7C15 ^ seed, 11
    state = DropoutState(key, step)
    drop = Dropout(state, rate, 3) if rate else None
    path = Dropout(state, path_rate, 4) if path_rate else None
    d64 = (key, step, 3, rate) if rate else None
    p64 = (key, step, 4, path_rate) if path_rate else None
    return case, par, par64, drop, path, d64, p64


ALL = ("post_gamma", "post_beta", "scale", "gate", "pre_gamma", "pre_beta")
PRESENT = [ALL, (), ("scale", "pre_gamma"), ("gate", "post_gamma"), ("post_beta", "pre_beta", "scale")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,pre", JOINS)
@pytest.mark.parametrize("channels", [8, 56, 96, 168, 256, 376, 512, 648, 1024, 1600, 2056, 2560, 3848, 5128, 8192])
def test_join(channels, post, pre, dtype):
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    join = ResidualJoin(channels, post, pre, 1e-5, dtype)
    for k, (b, t) in enumerate([(1, 1), (3, 45), (2, 311)]):
        seed = channels + 7 * k + 31 * JOINS.index((post, pre))
        present = PRESENT[(seed + k) % 5] if k else ALL
        rate, path_rate = [(0.1, 0.4), (0.0, 0.0), (0.3, 0.0)][(k + channels // 8) % 3]
        case, par, par64, drop, path, d64, p64 = join_case(seed, b, t, channels, dtype, post, pre, present, rate, path_rate)
        (x, x64), (z, z64), (dy, dy64), (dh, dh64) = (case[n] for n in ("x", "z", "dy", "dh"))
        y, h = join.forward(x, z, **par, drop=drop, path=path)
        y64, _ = ref.join_fwd(x64, z64, post, pre, 1e-5, par64, d64, p64)
        d, p, s, g = ref.join_weights(x64.shape, par64["scale"], par64["gate"], d64, p64)
        w = d * p * (s * g).abs()
        _, rz = ref.stats(z64, post, 1e-5) if post != "none" else (0, 1.0)
        gm = par64["post_gamma"].abs() if par64["post_gamma"] is not None else 1.0
        bt = par64["post_beta"].abs() if par64["post_beta"] is not None else 0.0
        size = x64.abs() + w * ((z64.abs() + z64.abs().mean(-1, keepdim=True)) * rz * gm + bt)
        close("y", y, y64, size, OPS, half_step(dtype))
        assert (h is None) == (pre == "none")
        stored = y.double().cpu()  # h and the backward are those of y as stored
        if h is not None:
            want = ref.norm_fwd(stored, pre, 1e-5, par64["pre_gamma"], par64["pre_beta"])
            _, ry = ref.stats(stored, pre, 1e-5)
            gp = par64["pre_gamma"].abs() if par64["pre_gamma"] is not None else 1.0
            bp = par64["pre_beta"].abs() if par64["pre_beta"] is not None else 0.0
            close("h", h, want, (stored.abs() + stored.abs().mean(-1, keepdim=True)) * ry * gp + bp, OPS, half_step(dtype))
        use_dy, use_dh = (k != 1 or pre == "none"), pre != "none" and k != 2
        got = join.backward(y, z, dy if use_dy else None, dh if use_dh else None, **par, drop=drop, path=path)
        grad, size = ref.join_bwd(stored, z64, dy64 if use_dy else None, dh64 if use_dh else None, post, pre, 1e-5, par64,
                                  d64, p64)
        c = cond(stored, pre).max() if pre != "none" else 1.0
        c = max(float(c), float(cond(z64, post).max()) if post != "none" else 1.0)
        for n, v in got._asdict().items():
            if n in ("dx", "dz"):
                close(n, v, grad[n], size[n], 2 * c * OPS, half_step(dtype))
                continue
            assert (v is None) == (par[n[1:]] is None), n
            if v is not None and n not in grad:  # no gradient reached h
                assert not v.any(), n
            elif v is not None:
                close(n, v, grad[n], size[n], 2 * c * OPS + LONG)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 100003])
def test_dropout(n, dtype):
    """The decisions are exact: what is kept is x / kept rounded once (fp32: twice), the rest 0."""
    import numpy as np
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, apply_dropout
    gen = torch.Generator().manual_seed(n)
    x, x64 = make(gen, (n,), dtype)
    state = DropoutState(2**63 + n, 2**32 + 5)  # the step counts modulo 2^32
    for rate, span in ((0.1, 1), (0.5, 8), (0.3, 24), (65535 / 65536, 1), (0.25, 3), (0.4, 10**6), (0.3, 2), (0.3, 7), (0.3, 9), (0.2, 1001)):
        for site in (0, 2**32 - 1):
            got = apply_dropout(x, Dropout(state, rate, site), span).double().cpu()
            keep = torch.from_numpy(ref.keep(np.arange(n) // span, 2**63 + n, 5, site, rate))
            want = x64 * ref.kept_scale(rate)
            assert not got[~keep].any()
            assert ((got - want).abs()[keep] <= (half_step(dtype) + 2 * 2.0**-24) * want.abs()[keep]).all()
    assert torch.equal(apply_dropout(x, None), x) and torch.equal(apply_dropout(x, Dropout(state, 0.0, 1)), x)


def test_dropped_infinities_and_nan_are_zero_kept_ones_stay():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, apply_dropout
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    drop = Dropout(DropoutState(5), 0.5, 1)
    ones = torch.ones(1, 4, 256, device="cuda")
    keep = apply_dropout(ones, drop) != 0
    for v in (float("nan"), float("inf"), -float("inf")):
        y = apply_dropout(ones * v, drop)
        assert (y[~keep] == 0).all()
        assert (torch.isnan(y) if v != v else y == v)[keep].all()
        y, _ = ResidualJoin(256, dtype="f32").forward(ones, ones * v, drop=drop)
        assert (y[~keep] == 1).all() and (torch.isnan(y) if v != v else y == v)[keep].all()


def test_a_row_of_nan_or_zeros_stays_in_its_row():
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm
    for kind in ("layer", "rms"):
        x = torch.randn(1, 9, 96, device="cuda")
        clean = BlockNorm(96, kind, dtype="f32").forward(x)
        x[0, 3] = float("nan")
        x[0, 5] = 0
        h = BlockNorm(96, kind, dtype="f32").forward(x)
        rest = [r for r in range(9) if r not in (3, 5)]
        assert torch.equal(h[0, rest], clean[0, rest]) and torch.isnan(h[0, 3]).all() and not h[0, 5].any()


def test_no_rows():
    from shifted_window_attention_cyclic_gb300.dropout import apply_dropout
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    g, gate = torch.ones(64, device="cuda"), torch.ones(2, 64, device="cuda")
    for shape in ((2, 0, 64), (2, 3, 0, 64)):
        x = torch.empty(shape, device="cuda")
        dx, dg, db = BlockNorm(64, dtype="f32").backward(x, x, g, g)
        assert dx.shape == x.shape and not dg.any() and not db.any()
        j = ResidualJoin(64, "rms", "layer", dtype="f32")
        y, h = j.forward(x, x, g, g, g, gate, g, g)
        out = j.backward(x, x, x, x, g, g, g, gate, g, g)
        assert y.shape == h.shape == x.shape and all(not t.any() for t in out)
        assert apply_dropout(x, None).shape == x.shape
    x, none = torch.empty((0, 5, 64), device="cuda"), torch.empty(0, 64, device="cuda")
    out = ResidualJoin(64, "rms", "layer", dtype="f32").backward(x, x, x, x, g, g, g, none, g, g)
    assert out.dgate.shape == (0, 64) and not out.dscale.any()


def test_in_place_and_same_bits_again():
    from shifted_window_attention_cyclic_gb300.dropout import apply_dropout
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    case, par, _, drop, path, _, _ = join_case(3, 2, 5000, 384, "bf16", "layer", "rms", ALL, 0.2, 0.3)
    x, z, dy, dh = (case[n][0] for n in ("x", "z", "dy", "dh"))
    join = ResidualJoin(384, "layer", "rms")
    y, h = join.forward(x, z, **par, drop=drop, path=path)
    first = join.backward(y, z, dy, dh, **par, drop=drop, path=path)
    for _ in range(3):
        again = join.backward(y, z, dy, dh, **par, drop=drop, path=path)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    x2, z2 = x.clone(), z.clone()
    y2, h2 = join.forward(x2, z2, **par, drop=drop, path=path, y=x2, h=z2)
    assert y2 is x2 and torch.equal(y2, y) and torch.equal(h2, h)
    norm = BlockNorm(384)
    assert torch.equal(norm.forward(x.clone(), h=None), norm.forward(x))
    x3 = x.clone()
    assert torch.equal(norm.forward(x3, h=x3), norm.forward(x))
    dx = norm.backward(x, dy, dres=dh)[0]
    dy2 = dy.clone()
    assert torch.equal(norm.backward(x, dy2, dres=dh, dx=dy2)[0], dx)
    x4 = x.clone()
    assert torch.equal(apply_dropout(x4, drop, out=x4), apply_dropout(x, drop))


def test_tensors_on_16_byte_boundaries():
    """The contract asks for 16 bytes: fp32 tensors 16 off a 32-byte boundary give the same bits as aligned ones."""
    from shifted_window_attention_cyclic_gb300.dropout import apply_dropout
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    for c in (40, 256, 1032):
        case, par, _, drop, path, _, _ = join_case(c, 2, 77, c, "f32", "layer", "rms", ALL, 0.2, 0.3)
        x, z, dy, dh = (case[n][0] for n in ("x", "z", "dy", "dh"))

        def off(t):
            flat = torch.empty(t.numel() + 4, device="cuda", dtype=t.dtype)[4:].view(t.shape)
            assert flat.data_ptr() % 32 == 16
            return flat.copy_(t)

        join, norm = ResidualJoin(c, "layer", "rms", dtype="f32"), BlockNorm(c, dtype="f32")
        y, h = join.forward(x, z, **par, drop=drop, path=path)
        y2, h2 = join.forward(off(x), off(z), **par, drop=drop, path=path, y=off(x), h=off(x))
        assert torch.equal(y, y2) and torch.equal(h, h2)
        a, b = (join.backward(f(y), f(z), f(dy), f(dh), **par, drop=drop, path=path) for f in (lambda t: t, off))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert torch.equal(norm.forward(x), norm.forward(off(x), h=off(x)))
        assert torch.equal(norm.backward(x, dy)[0], norm.backward(off(x), off(dy), dx=off(x))[0])
        assert torch.equal(apply_dropout(x, drop), apply_dropout(off(x), drop, out=off(x)))


def test_other_stream_and_captured():
    """A backward on a side stream while another runs on the current one, and a
    captured step whose replays take the state's step."""
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    case, par, _, drop, path, _, _ = join_case(4, 2, 3000, 256, "bf16", "rms", "layer", ALL, 0.2, 0.3)
    x, z, dy, dh = (case[n][0] for n in ("x", "z", "dy", "dh"))
    join = ResidualJoin(256, "rms", "layer")
    kw = dict(par, drop=drop, path=path)

    def step():
        y, h = join.forward(x, z, **kw)
        return (y, h) + tuple(join.backward(y, z, dy, dh, **kw))

    want = {}
    for k in range(3):
        want[k] = [t.clone() for t in step()]
        drop.state.advance()
    drop.state.tensor[1] -= 3
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h = join.forward(x, z, **kw, stream=side)
    here = step()
    there = join.backward(y, z, dy, dh, **kw, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, h) + tuple(there), want[0]))
    assert all(torch.equal(a, b) for a, b in zip(here, want[0]))
    graphs = []
    for _ in range(2):  # two graphs: each keeps its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for k in range(3):
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))
        drop.state.advance()


def test_many_images_with_gates():
    """More images than CTAs, and images that end inside and with a CTA's rows."""
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    for b, t, c in ((700, 1, 64), (900, 3, 32), (5, 997, 64), (304, 8, 256)):
        case, par, par64, drop, path, d64, p64 = join_case(b, b, t, c, "f32", "layer", "none", ALL, 0.1, 0.3)
        (y, y64), (z, z64), (dy, dy64), _ = (case[n] for n in ("x", "z", "dy", "dh"))
        got = ResidualJoin(c, "layer", "none", dtype="f32").backward(y, z, dy, None, **par, drop=drop, path=path)
        grad, size = ref.join_bwd(y64, z64, dy64, None, "layer", "none", 1e-5, par64, d64, p64)
        k = float(cond(z64, "layer").max())
        for n in ("dgate", "dscale", "dpost_gamma", "dpost_beta"):
            close(n, getattr(got, n), grad[n], size[n], 2 * k * OPS + LONG)


def test_difference_quotients():
    """The kernels' own forward moves by the kernels' gradient: fp32, a step of
    1e-2 along a random direction. The quotient's error: the loss is a sum of
    about 5e4 terms of order 1 rounded to 2^-24 each (random signs: 5e4^.5 *
    2^-24 / 2e-2 = 7e-4, times about 10 for the row statistics) and the third
    derivative times 1e-4 / 6, which the bound takes as 1e-3 of the gradient's
    own norm along the step."""
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    case, par, _, drop, path, _, _ = join_case(12, 2, 97, 256, "f32", "layer", "rms", ALL, 0.2, 0.3)
    x, z, dy, dh = (case[n][0] for n in ("x", "z", "dy", "dh"))
    join = ResidualJoin(256, "layer", "rms", dtype="f32")

    def loss(x, z, par):
        y, h = join.forward(x, z, **par, drop=drop, path=path)
        return float((y.double() * dy).sum() + (h.double() * dh).sum())

    y, _ = join.forward(x, z, **par, drop=drop, path=path)
    got = join.backward(y, z, dy, dh, **par, drop=drop, path=path)._asdict()
    gen = torch.Generator().manual_seed(5)
    for name in ["dx", "dz"] + ["d" + n for n in ALL]:
        t = {"dx": x, "dz": z}.get(name, par.get(name[1:]))
        step = torch.randn(t.shape, generator=gen).cuda()
        moved = []
        for sign in (1, -1):
            new = t + sign * 1e-2 * step
            moved.append(loss(new if name == "dx" else x, new if name == "dz" else z,
                              {n: (new if "d" + n == name else p) for n, p in par.items()}))
        quotient, want = (moved[0] - moved[1]) / 2e-2, float((got[name].double() * step).sum())
        assert abs(quotient - want) <= 7e-3 + 1e-3 * float((got[name].double() * step).norm()) * 10, name


def test_a_block_trains_through_all_of_them():
    """norm -> projections -> window attention with dropout -> projection -> join -> dropout, as a training step uses
    them, against autograd over the 64-bit formulas."""
    import numpy as np
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, dropout
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention, swin_window_attention
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin, block_norm, residual_join
    grid, heads, c, b = (9, 13), 2, 64, 2
    attn = SwinWindowAttention(grid, (4, 4), (2, 2), (0, 1), heads, 32, b, "f32")
    state = DropoutState(77, 5)
    drops = [Dropout(state, 0.2, s) for s in range(4)]
    gen = torch.Generator().manual_seed(8)
    shape = (b,) + grid + (c,)
    leaf = {"x": torch.randn(shape, generator=gen), "wq": torch.randn(c, 3 * c, generator=gen) / 8,
            "wo": torch.randn(c, c, generator=gen) / 8, "bias": torch.randn(attn.bias_shape, generator=gen) * 0.1}
    for n in ("g1", "b1", "g2", "b2", "g3", "scale"):
        leaf[n] = torch.randn(c, generator=gen) * 0.2 + 0.8
    leaf["gate"] = torch.randn(b, c, generator=gen) * 0.2 + 0.8
    dy, dh = torch.randn(shape, generator=gen), torch.randn(shape, generator=gen)

    p = {n: t.cuda().requires_grad_(True) for n, t in leaf.items()}
    h = block_norm(BlockNorm(c, "layer", dtype="f32"), p["x"], p["g1"], p["b1"])
    q, k, v = (h @ p["wq"]).chunk(3, -1)
    o = swin_window_attention(attn, q, k, v, p["bias"], dropout=drops[0])
    y, h2 = residual_join(ResidualJoin(c, "rms", "layer", dtype="f32"), p["x"], o @ p["wo"], p["g3"], None, p["scale"],
                          p["gate"], p["g2"], p["b2"], drops[1], drops[2])
    out = dropout(h2, drops[3])
    ((y * dy.cuda()).sum() + (out * dh.cuda()).sum()).backward()
    assert C.swin_attn_status(attn.plan) == 0

    r = {n: t.double().requires_grad_(True) for n, t in leaf.items()}
    tables = C.swin_attn_plan_tables(attn.plan)[:2] + (C.swin_attn_plan_tables(attn.plan)[3],)
    flat = lambda t: t.reshape(b, -1, t.shape[-1])  # noqa: E731
    key = lambda s: (77, 5, s, 0.2)  # noqa: E731
    h64 = ref.norm_fwd(r["x"], "layer", 1e-5, r["g1"], r["b1"])
    q, k, v = (flat(h64) @ r["wq"]).chunk(3, -1)
    o64 = ref.attn(q, k, v, r["bias"], None, tables, heads, key(0))["o"]
    y64, h264 = ref.join_fwd(flat(r["x"]), o64 @ r["wo"], "rms", "layer", 1e-5,
                             dict(post_gamma=r["g3"], scale=r["scale"], gate=r["gate"], pre_gamma=r["g2"], pre_beta=r["b2"]),
                             key(1), key(2))
    w = torch.from_numpy(ref.weights(int(np.prod(shape)), 1, key(3))).view(h264.shape)
    ((y64 * flat(dy)).sum() + (h264 * w * flat(dh)).sum()).backward()
    # fp32 throughout: a chain of five stages, each with relative error below OPS of its norm
    for n in leaf:
        e = (p[n].grad.double().cpu() - r[n].grad).norm() / r[n].grad.norm()
        assert e <= 5 * OPS, (n, float(e))
    assert (y.double().cpu().view(y64.shape) - y64).norm() <= 5 * OPS * y64.norm()

    # second derivatives are refused, not wrong
    x = torch.randn(1, 3, 64, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(block_norm(BlockNorm(64, dtype="f32"), x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        g.sum().backward()

    # a state advanced between the forward and the backward is an error, not a wrong gradient
    out = dropout(p["x"], drops[0])
    state.advance()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_python_refuses_what_the_library_cannot_see():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, apply_dropout
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    x = torch.zeros(2, 4, 6, 64, device="cuda", dtype=torch.bfloat16)
    g, gate = torch.ones(64, device="cuda"), torch.ones(2, 64, device="cuda")
    norm, join = BlockNorm(64), ResidualJoin(64, "none", "layer")
    for match, call in (
            ("dtype", lambda: norm.forward(x.float())),
            ("shape", lambda: norm.forward(x[..., :32].contiguous())),
            ("contiguous", lambda: norm.forward(x.transpose(1, 2))),
            ("aligned", lambda: norm.forward(torch.zeros(65, device="cuda", dtype=torch.bfloat16)[1:].view(1, 64))),
            ("gamma", lambda: norm.forward(x, g[:32])),
            ("gamma", lambda: norm.forward(x, g.double())),
            ("beta", lambda: norm.forward(x, g, g.cpu())),
            ("shape", lambda: norm.backward(x, x[:1])),
            ("dh", lambda: norm.backward(x, None)),
            ("dx", lambda: norm.backward(x, x, dx=x.float())),
            ("post_gamma", lambda: join.forward(x, x, post_gamma=g)),
            ("gate", lambda: join.forward(x, x, gate=g)),
            ("gate", lambda: join.forward(x, x, gate=gate.t().contiguous().t())),
            ("z", lambda: join.forward(x, None)),
            ("drop", lambda: join.forward(x, x, drop=0.1)),
            ("drop: its state", lambda: join.forward(x, x, drop=Dropout(DropoutState(1, device="cpu"), 0.1, 0))),
            ("dy, dh", lambda: join.backward(x, x, None, None)),
            ("dh", lambda: ResidualJoin(64).backward(x, x, x, x)),
            ("h: the join", lambda: ResidualJoin(64).forward(x, x, h=x)),
            ("span", lambda: apply_dropout(x, None, span=0)),
            ("out", lambda: apply_dropout(x, None, out=x.float()))):
        with pytest.raises(ValueError, match=match):
            call()
