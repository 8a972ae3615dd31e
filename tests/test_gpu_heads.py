"""Head norm and rotary positions on the GPU against the 64-bit reference, over
head sizes, layouts, types, strides and positions.

Tolerances. A head's statistics come from 8 values a lane and at most 5 shuffles
twice, and a value passes about as many roundings again on the way out: OPS = 64
roundings of 2^-24 bound the relative error of what a head computes, times the
size of what it was summed from. An angle is off by half a step of a float below
one half turn (pi 2^-25) and by what its 64 bits leave out, a cosine or sine by
two steps more (sincospif, 2 ulp): under 2^-22 in all, and again a step for the
amplitude, so TURN = 2^-21 of the size. Parameter gradients add up to LONG more
roundings (the items of a thread, then the fold). bf16 outputs add half a step,
2^-8 of the value."""
import gc

import pytest

torch = pytest.importorskip("torch")

from tests import heads_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def no_memory_kept():
    """Give the allocator's blocks back: a later test counts what its calls hold, and a cached block may be the larger one."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


OPS, TURN, LONG = 64 * 2.0**-24, 2.0**-21, 256 * 2.0**-24
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0**-8, "f32": 2.0**-24}


def close(name, got, want, size, fp32, store=2.0**-24):
    got = got.double().cpu().reshape(want.shape)
    bound = fp32 * size + store * want.abs() + 1e-30
    assert torch.isfinite(got).all(), name
    bad = ((got - want).abs() - bound).max() if want.numel() else torch.tensor(-1.0)
    assert bad <= 0, "%s: over the bound by %.3e (error %.3e)" % (name, bad, (got - want).abs().max())


def make(gen, shape, dtype, std=1.0, mean=0.0):
    t = (torch.randn(shape, generator=gen) * std + mean).to(TDT[dtype])
    return t.cuda(), t.double()


def check(gen, spec, images, grid, packed=True, positions=None, gammas=True, betas=True):
    """Forward and backward of one call against the reference."""
    lead, hd, dtype = (images,) + tuple(grid), spec.head_dim, spec.dtype
    qkv, qkv64 = make(gen, lead + (spec.q_width + 2 * spec.kv_width,), dtype, 1.5, 0.4)
    x, x64 = spec.split(qkv), spec.split(qkv64)
    if not packed:
        x = [t.contiguous() for t in x]
    par, par64 = {}, {}
    for side in "qk":
        for name, some, std, mean in (("gamma", gammas, 0.3, 1.0), ("beta", betas, 0.3, 0.0)):
            t = torch.randn(hd, generator=gen) * std + mean if some and spec.norm != "none" else None
            par["%s_%s" % (side, name)] = None if t is None else t.cuda()
            par64["%s_%s" % (side, name)] = None if t is None else t.double()
    rot, t = spec.rotary, None
    if rot is not None:
        at = ref.grid_positions(images, grid) if positions is None else positions.cpu().reshape(
            (images, -1, rot.axes) if positions.numel() == images * torch.Size(grid).numel() * rot.axes else (1, -1, rot.axes))
        t = ref.turns(at, rot.frequencies, rot.axis_of)
    layout, amplitude = ("half", 1.0) if rot is None else (rot.layout, rot.amplitude)
    split = lambda u: u.reshape(images, -1, u.shape[-1] // hd, hd)  # noqa: E731
    out = spec.forward(*x, **par, positions=positions)
    douts = [make(gen, o.shape, dtype) for o in out]
    g = spec.backward(*[d for d, _ in douts], x[0], x[1], **par, positions=positions, packed=packed)
    for i, side in enumerate("qk"):
        want, size = ref.heads_fwd(split(x64[i]), t, layout, amplitude, spec.norm, spec.eps, par64[side + "_gamma"],
                                   par64[side + "_beta"])
        assert out[i].is_contiguous()
        close(side, out[i], want, size, OPS + TURN, HALF[dtype])
        want, size = ref.heads_bwd(split(x64[i]), split(douts[i][1]), t, layout, amplitude, spec.norm, spec.eps,
                                   par64[side + "_gamma"])
        close("d" + side, g[i], want[0], size[0], OPS + TURN, HALF[dtype])
        for k, name in ((1, "gamma"), (2, "beta")):
            got = getattr(g, "d%s_%s" % (side, name))
            assert (got is None) == (par["%s_%s" % (side, name)] is None)
            if got is not None:
                close("d%s_%s" % (side, name), got, want[k], size[k], OPS + TURN + LONG)
    assert torch.equal(out[2], x[2]) and torch.equal(g.dv, douts[2][0])
    if packed:
        assert g.dqkv.is_contiguous() and torch.equal(g.dqkv, torch.cat([g.dq, g.dk, g.dv], -1))


HEAD_DIMS = [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", HEAD_DIMS)
def test_head_sizes(hd, dtype):
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(hd)
    cases = [((1,), 1, 1, 1), ((37,), 2, 3, 3), ((3, 7), 3, 8, 2), ((2, 5, 9), 1, 1, 4), ((11, 13), 2, 5, 1)]
    for k, (grid, images, heads, kv) in enumerate(cases):
        rot = 16 * (1 + (hd // 16 + 3 * k) % (hd // 16))
        rotary = Rotary(min(rot, hd), axes=len(grid), layout=("half", "interleaved")[(k + hd // 16) % 2],
                        amplitude=(1.0, 1.25)[k % 2]) if k != 3 or hd == 16 else Rotary(hd, axes=len(grid))
        spec = AttentionHeads(heads, hd, rotary, ("rms", "layer", "none")[(k + hd // 16) % 3], 1e-5, dtype, kv)
        check(gen, spec, images, grid, packed=k % 2 == 0, gammas=k != 1, betas=k in (0, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("layout", ["half", "interleaved", None])
def test_layouts_and_norms(layout, norm, dtype):
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(7)
    for hd, rot, axes, grid in ((32, 32, 2, (19, 23)), (32, 16, 3, (2, 5, 31)), (128, 64, 2, (9, 17)), (16, 16, 1, (300,))):
        rotary = Rotary(rot, axes, layout) if layout else None
        check(gen, AttentionHeads(4, hd, rotary, norm, 1e-5, dtype), 2, grid)


def test_many_tiles():
    """More tiles than CTAs: each walks several, with heads that do not divide a tile."""
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(8)
    for heads, kv, hd, dtype in ((7, 3, 32, "bf16"), (3, 1, 48, "f32"), (1, 1, 16, "bf16")):
        spec = AttentionHeads(heads, hd, Rotary(16, 2), "layer", 1e-5, dtype, kv)
        check(gen, spec, 2, (61, 1023), packed=heads != 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_many_heads(dtype):
    """More heads than a CTA takes at a time: a row in chunks, the last one ragged."""
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(14)
    for heads, kv, hd in ((64, 25, 256), (1024, 1, 16), (100, 13, 160)):
        spec = AttentionHeads(heads, hd, Rotary(16, 1), "rms", 1e-5, dtype, kv)
        check(gen, spec, 1, (19,))


def test_large_mean():
    """Heads far from zero: the mean is taken out before the squares."""
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads
    x = (torch.randn(1, 50, 64, generator=torch.Generator().manual_seed(1)) + 1000).cuda()
    y = AttentionHeads(2, 32, None, "layer", dtype="f32").forward(x)[0]
    want, size = ref.heads_fwd(x.double().cpu().view(1, 50, 2, 32), None, "half", 1.0, "layer", 1e-5)
    close("q", y, want, size, OPS)


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_given_positions(kind):
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(9)
    near = 2**31 - 1 if kind == torch.int32 else 2**45
    spec = AttentionHeads(4, 64, Rotary(64), "rms", dtype="f32", kv_heads=2)
    for shape in ((3, 1), (3, 29), (29,), (3, 29, 1)):
        at = torch.randint(-near, near, shape, generator=gen).to(kind).cuda()
        at.view(-1)[0] = 0
        check(gen, spec, 3, (shape[1] if len(shape) > 1 else shape[0],), positions=at)
    three = AttentionHeads(2, 32, Rotary(32, 3, "interleaved"), dtype="bf16")
    check(gen, three, 2, (5, 6), positions=torch.randint(-50, 5000, (2, 5, 6, 3), generator=gen).to(kind).cuda())
    check(gen, three, 2, (31,), positions=torch.randint(-50, 5000, (31, 3), generator=gen).to(kind).cuda())
    # the grid's own coordinates, given
    spec2 = AttentionHeads(2, 32, Rotary(32, 2))
    x = torch.randn(2, 7, 9, 64, generator=gen).to(torch.bfloat16).cuda()
    at = ref.grid_positions(1, (7, 9)).view(7, 9, 2).to(kind).contiguous().cuda()
    assert torch.equal(spec2.forward(x)[0], spec2.forward(x, positions=at)[0])


def test_scaled_rotaries():
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(10)
    at = torch.randint(0, 10**6, (2, 40), generator=gen).cuda()
    for rotary in (Rotary(64, scaling="linear", factor=8.0), Rotary(64, scaling="ntk", factor=8.0, layout="interleaved"),
                   Rotary(64, scaling="yarn", factor=32.0, trained=8192),
                   Rotary(64, frequencies=[1.7 ** -j for j in range(31)] + [-9.5], amplitude=-0.5)):
        check(gen, AttentionHeads(2, 64, rotary, dtype="f32"), 2, (40,), positions=at)


def test_a_token_alone_is_the_token_among_others():
    """One token of each request, as a decoder calls it: the bits of the whole sequence's call."""
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(11)
    spec = AttentionHeads(16, 128, Rotary(128), "rms", kv_heads=4)
    q, k = torch.randn(5, 33, 2048, generator=gen).bfloat16().cuda(), torch.randn(5, 33, 512, generator=gen).bfloat16().cuda()
    qg, kg = torch.randn(128, generator=gen).cuda(), torch.randn(128, generator=gen).cuda()
    whole = spec.forward(q, k, q_gamma=qg, k_gamma=kg)
    for t in (0, 7, 32):
        at = torch.full((5, 1), t, device="cuda")
        one = spec.forward(q[:, t:t + 1].contiguous(), k[:, t:t + 1].contiguous(), q_gamma=qg, k_gamma=kg, positions=at)
        assert torch.equal(one[0], whole[0][:, t:t + 1]) and torch.equal(one[1], whole[1][:, t:t + 1])
        view = spec.forward(q[:, t:t + 1], k[:, t:t + 1], q_gamma=qg, k_gamma=kg, positions=at)  # rows 33 apart
        assert torch.equal(view[0], one[0]) and torch.equal(view[1], one[1])


def test_in_place_and_views():
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    gen = torch.Generator().manual_seed(12)
    for dtype in ("bf16", "f32"):
        spec = AttentionHeads(4, 32, Rotary(32, 2), "rms", dtype=dtype)
        qkv = torch.randn(2, 9, 40, 384, generator=gen).to(TDT[dtype]).cuda()
        before = qkv.clone()
        q, k, v = spec.split(qkv)
        want = spec.forward(q, k, v)
        wide = torch.full((2, 9, 40, 512), 7.0, dtype=TDT[dtype], device="cuda")  # outputs inside wider rows
        spec.forward(q, k, v, q_out=wide[..., 16:144], k_out=wide[..., 160:288], v_out=wide[..., 384:])
        assert torch.equal(qkv, before)
        for o, at in zip(want, (16, 160, 384)):
            assert torch.equal(wide[..., at:at + 128], o)
        for a, b in ((0, 16), (144, 160), (288, 384)):
            assert (wide[..., a:b] == 7.0).all()
        spec.forward(q, k, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before[..., 256:])
        with pytest.raises(Exception):
            spec.forward(q, k, q_out=k, k_out=q)
        # fp32 rows that start on 16 bytes, not on 32
        if dtype == "f32":
            x = torch.empty(720 * 132 + 4, device="cuda")[4:].view(2, 9, 40, 132)[..., :128]
            x.copy_(before[..., :128])
            assert x.data_ptr() % 32 == 16 and torch.equal(spec.forward(x)[0], want[0])


def test_rows_past_32_bit_offsets():
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    spec = AttentionHeads(16, 128, Rotary(128), "rms")
    rows = 780_000  # 780 000 x 6144 values: 2^32 and more, 9.6 GB
    qkv = torch.empty(1, rows, 6144, dtype=torch.bfloat16, device="cuda")
    qkv.normal_()
    out = spec.forward(*spec.split(qkv))
    at = torch.tensor([0, 1, 349525, 349526, 699050, 699051, rows - 1], device="cuda")
    few = spec.forward(*spec.split(qkv[:, at].contiguous()), positions=at[None])
    for a, b in zip(out, few):
        assert torch.equal(a[:, at], b)
    del out
    g = spec.backward(*spec.split(qkv), *spec.split(qkv)[:2], packed=True)
    few_in = qkv[:, at].contiguous()
    few = spec.backward(*spec.split(few_in), *spec.split(few_in)[:2], positions=at[None], packed=True)
    assert torch.equal(g.dqkv[:, at], few.dqkv)


def test_no_rows():
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    spec = AttentionHeads(2, 32, Rotary(32, 2), "layer")
    gamma, beta = torch.ones(32, device="cuda"), torch.ones(32, device="cuda")
    x = torch.empty(2, 0, 5, 192, dtype=torch.bfloat16, device="cuda")
    out = spec.forward(*spec.split(x), q_gamma=gamma, k_beta=beta)
    assert all(o.shape == (2, 0, 5, 64) for o in out)
    g = spec.backward(*out, *spec.split(x)[:2], q_gamma=gamma, k_beta=beta, packed=True)
    assert g.dqkv.shape == x.shape and (g.dq_gamma == 0).all() and (g.dk_beta == 0).all()


def test_same_bits_every_run():
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    spec = AttentionHeads(8, 32, Rotary(32, 2), "rms")
    qkv, gamma = torch.randn(2, 90, 180, 768, device="cuda").bfloat16(), torch.ones(32, device="cuda")
    d = spec.forward(*spec.split(qkv), q_gamma=gamma, k_gamma=gamma)
    runs = [spec.backward(*d, *spec.split(qkv)[:2], q_gamma=gamma, k_gamma=gamma, packed=True) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(getattr(r, n), getattr(runs[0], n)) for n in ("dqkv", "dq_gamma", "dk_gamma"))


def test_streams_and_graphs():
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    spec = AttentionHeads(8, 32, Rotary(32, 2), "rms")
    gamma = [torch.randn(32, device="cuda") for _ in range(2)]
    xs = [torch.randn(1, 64, 128, 768, device="cuda").bfloat16() for _ in range(2)]

    def step(x, stream=None):
        out = spec.forward(*spec.split(x), q_gamma=gamma[0], k_gamma=gamma[1], stream=stream)
        return spec.backward(*out, *spec.split(x)[:2], q_gamma=gamma[0], k_gamma=gamma[1], packed=True, stream=stream)

    want = [step(x) for x in xs]
    side = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[step(x, s) for x, s in zip(xs, side)] for _ in range(5)]
    torch.cuda.synchronize()
    names = ("dqkv", "dq_gamma", "dk_gamma")
    for pair in got:
        for g, w in zip(pair, want):
            assert all(torch.equal(getattr(g, n), getattr(w, n)) for n in names)
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x)
        graphs.append((graph, out))
    torch.cuda.synchronize()
    for _ in range(4):  # both at once
        for (graph, _), s in zip(graphs, side):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, g), w in zip(graphs, want):
        assert all(torch.equal(getattr(g, n), getattr(w, n)) for n in names)


@pytest.mark.parametrize("packed", [True, False])
def test_autograd(packed):
    from shifted_window_attention_cyclic_gb300 import heads as H
    gen = torch.Generator().manual_seed(13)
    spec = H.AttentionHeads(3, 32, H.Rotary(16, 2), "layer", dtype="f32")
    leaf = torch.randn(2, 5, 7, 288, generator=gen).cuda().requires_grad_(True)
    par = [(torch.randn(32, generator=gen) + 1).cuda().requires_grad_(True) for _ in range(4)]
    w = [torch.randn(2, 5, 7, 96, generator=gen).cuda() for _ in range(3)]

    def loss(leaf, par):
        out = H.attention_heads_packed(spec, leaf, *par) if packed else H.attention_heads(spec, *spec.split(leaf), *par)
        return sum((o * x).sum(dtype=torch.float64) for o, x in zip(out, w))

    loss(leaf, par).backward()
    # the passes that check() holds to the formula
    g = spec.backward(*w, *spec.split(leaf.detach())[:2], *[p.detach() for p in par], packed=True)
    assert torch.equal(leaf.grad, g.dqkv)
    assert all(torch.equal(p.grad, x) for p, x in zip(par, (g.dq_gamma, g.dq_beta, g.dk_gamma, g.dk_beta)))
    # a slice that starts anywhere, and a gradient that does
    flat = torch.cat([leaf.new_zeros(1), leaf.detach().flatten()]).requires_grad_(True)
    loss(flat[1:].view(leaf.shape), [p.detach() for p in par]).backward()
    assert torch.equal(flat.grad[1:].view(leaf.shape), leaf.grad)


def test_another_device_than_the_current():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
    spec = AttentionHeads(2, 32, Rotary(32, 1))
    x = torch.randn(1, 9, 64, device="cuda:1").bfloat16()
    assert spec.forward(x)[0].device == x.device
