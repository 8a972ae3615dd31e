"""AdamW over many tensors and the gradients' norm on the GPU against the 64-bit
reference.

Tolerances. m and v are sums of two products whose factors are fp32 roundings of
the betas, of the gradient and of the clipping factor: OPS = 8 roundings of 2^-24
of the terms' sizes. The clipping factor itself comes from a sum of squares, each
added to at most 16 others in fp32 and to the rest in fp64: NORM = 24 roundings.
The update m / (root / fix + eps) passes 8 more than m and root together (OPS each)
and the weight one more. bf16 parameters are the nearest to their master weights.
e4m3 values are nearest (half a step, 2^-4 of the value, 2^-10 of a scale for the
smallest) wherever the exact ratio is not within 2^-18 of a tie."""
import gc

import pytest

torch = pytest.importorskip("torch")

from tests import optim_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def no_memory_kept():
    """Give the allocator's blocks back: a later test counts what its calls hold, and a cached block may be the larger one."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


STEP = 2.0**-24
OPS, NORM = 8 * STEP, 24 * STEP
LR, DECAY, BETAS, EPS = 1e-2, 0.1, (0.9, 0.97), 1e-8


def near(name, got, want, bound):
    got = got.double().cpu().flatten()
    bad = ((got - want).abs() - bound - 1e-38).max() if want.numel() else torch.tensor(-1.0)
    assert torch.isfinite(got).all() and bad <= 0, "%s: over the bound by %.3e" % (name, bad)


def tensor(gen, n, dtype, std, off=0, mean=0.0):
    """n values that start `off` elements behind a 512-byte boundary."""
    t = torch.empty(n + off, dtype=dtype, device="cuda")[off:]
    t.copy_((torch.randn(n, generator=gen) * std + mean).to(dtype))
    return t


def check_states(opt, i, p, m1, v1, sm, slack, half_grad):
    """The 8-bit states of parameter i against the reference's values and scales."""
    o = opt._first[i]
    for name, q, scales, x, floor in (("m", opt.m, opt.m_scale, m1, False), ("v", opt.v, opt.v_scale, torch.sqrt(v1), True)):
        values, scale = ref.to_e4m3(x, floor)
        u = slice(o // 256, o // 256 + scale.numel())
        near(name + " scale", scales[u], scale, (OPS + slack) * scale + (sm.max() / 448 if name == "m" else 0))
        got = q[o:o + p.numel()].double().cpu()
        each = scale.repeat_interleave(256)[:p.numel()]
        ratio = (x / torch.where(each > 0, each, 1.0)).abs()
        mid = (ref.E4M3[1:] + ref.E4M3[:-1]) / 2
        k = torch.searchsorted(mid, ratio.contiguous()).clamp(max=mid.numel() - 1)
        gap = torch.minimum((mid[k] - ratio).abs(), (mid[(k - 1).clamp(min=0)] - ratio).abs())
        # m's own error, in scales, can move a ratio too
        tie = gap <= 2.0**-18 * ratio + (2 * sm / each.clamp(min=1e-38) if name == "m" else 0.0)
        assert torch.equal(got[~tie], values[~tie]), name
        # what is left out stays few: a bf16 gradient has 8 significant bits, a tie 5 of which the last is set, so where the
        # largest of 256 has few bits itself, one in 2^4 values of a new state is an exact tie
        assert p.numel() < 1000 or tie.double().mean() <= (2.0**-3 if half_grad else 0.01)
        near(name + " near a tie", got[tie], ratio[tie] * torch.sign(values[tie]), 2.0**-4 * 1.001 * ratio[tie] + 2.0**-9)


def check_step(opt, grads, decays, max_norm=None):
    """One step, against the reference from the states as they are before it."""
    before = []
    for i, p in enumerate(opt.params):
        m, v = opt.moments(i)
        at = opt._master_at[i]
        w = p if at is None else opt.master[at:at + p.numel()]
        before.append([t.detach().double().cpu().flatten() for t in (w, m, v)])
    g64 = [None if g is None else g.double().cpu().flatten() for g in grads]
    t = int(opt.steps) + 1
    opt.step(grads)
    assert int(opt.steps) == t
    clip, slack = 1.0, 0.0
    if max_norm:
        size = torch.sqrt(sum((g * g).sum() for g in g64 if g is not None))
        near("norm", opt.grad_norm, size.view(1), NORM * size)
        clip, slack = min(1.0, max_norm / float(size)), NORM
    for i, p in enumerate(opt.params):
        w, m, v = before[i]
        at, o = opt._master_at[i], opt._first[i]
        held = (p if at is None else opt.master[at:at + p.numel()]).detach().flatten()
        if g64[i] is None:
            assert torch.equal(held.double().cpu(), w)
            continue
        g = g64[i] * clip
        w1, m1, v1 = ref.adamw(w, g, m, v, t, LR, decays[i], *BETAS, EPS)
        sm = (BETAS[0] * m.abs() + (1 - BETAS[0]) * g.abs()) * (OPS + slack)
        sv = (BETAS[1] * v + (1 - BETAS[1]) * g * g) * (OPS + 2 * slack)
        step = LR / (1 - BETAS[0] ** t) / (torch.sqrt(v1) / (1 - BETAS[1] ** t) ** 0.5 + EPS)
        near("w", held, w1, step * sm + step * m1.abs() * (2 * OPS + slack) + 3 * STEP * (w.abs() + w1.abs()))
        if at is not None:
            assert torch.equal(p.detach().flatten(), held.to(torch.bfloat16))
        if opt.state_bits == 32:
            near("m", opt.m[o:o + p.numel()], m1, sm)
            near("v", opt.v[o:o + p.numel()], v1, sv)
        elif p.numel():
            check_states(opt, i, p, m1, v1, sm, slack, grads[i].dtype == torch.bfloat16)


def group(seed, sizes, kinds, state_bits, max_norm=None, off=0, std=0.3):
    """An optimiser over tensors of these sizes, and a function that makes gradients for it."""
    from shifted_window_attention_cyclic_gb300.optim import AdamW
    gen = torch.Generator().manual_seed(seed)
    kinds = [kinds[i % len(kinds)] for i in range(len(sizes))]
    params = [tensor(gen, n, p, 1.0, off * (i % 3)) for i, (n, (p, g)) in enumerate(zip(sizes, kinds))]
    decays = [DECAY if i % 2 else 0.0 for i in range(len(sizes))]
    opt = AdamW([{"params": [p], "weight_decay": d} for p, d in zip(params, decays)], lr=LR, betas=BETAS, eps=EPS,
                state_bits=state_bits, max_norm=max_norm)

    def grads(some=lambda i: True):
        return [tensor(gen, n, g, std * (1 + i % 4), off * ((i + 1) % 3)) if some(i) else None
                for i, (n, (p, g)) in enumerate(zip(sizes, kinds))]

    return opt, grads, decays


B, F = torch.bfloat16, torch.float32
KINDS = {"f32": [(F, F)], "bf16": [(B, B)], "mixed": [(F, F), (B, B), (B, F), (F, B)]}
SIZES = [1, 2, 7, 255, 256, 257, 511, 512, 1000, 4096, 5003, 0, 70001, 33, 256 * 9]


@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("kinds", sorted(KINDS))
@pytest.mark.parametrize("bits", [32, 8])
def test_steps(bits, kinds, off):
    """The first steps of new states, with and without clipping; tensors that start anywhere."""
    for max_norm in (None, 1.0):
        opt, grads, decays = group(1, SIZES, KINDS[kinds], bits, max_norm, off)
        for k in range(3):
            check_step(opt, grads(lambda i: k != 1 or i % 5 != 2), decays, max_norm)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [24, 25, 64, 65, 400, 401, 1024, 1025])
def test_many_tensors(count, bits):
    """Around what one table of tensors holds."""
    opt, grads, decays = group(2, [1 + (37 * i) % 700 for i in range(count)], KINDS["mixed"], bits, 2.0)
    for _ in range(2):
        check_step(opt, grads(), decays, 2.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_units(bits):
    """More units than warps: each walks several, across tensors."""
    opt, grads, decays = group(3, [1_500_001, 3, 2_000_000, 999_999], KINDS["mixed"], bits, 0.5)
    for _ in range(2):
        check_step(opt, grads(), decays, 0.5)


def test_small_gradients_keep_their_denominators():
    """In 8 bits a tiny second moment beside a large one is held above zero: no step grows past lr."""
    from shifted_window_attention_cyclic_gb300.optim import AdamW
    p = torch.zeros(512, device="cuda")
    opt = AdamW([p], lr=1.0, betas=(0.9, 0.9), eps=1e-8, weight_decay=0.0, state_bits=8)
    g = torch.full((512,), 1e-6, device="cuda")
    g[::256] = 100.0
    last = p.clone()
    for _ in range(20):
        opt.step([g])
        # |m| / sqrt(v) is 1 for a constant gradient; m and the root are off by up to 2^-4 each, a floored root is larger
        assert (p - last).abs().max() <= (1 + 2.0**-4) / (1 - 2.0**-4)
        last = p.clone()
    assert (opt.moments(0)[1] > 0).all()


def test_zero_gradients():
    from shifted_window_attention_cyclic_gb300.optim import AdamW
    for bits in (32, 8):
        p = torch.ones(300, device="cuda")
        opt = AdamW([p], lr=0.1, weight_decay=0.5, state_bits=bits, max_norm=1.0)
        opt.step([torch.zeros_like(p)])
        assert torch.allclose(p, torch.full_like(p, 0.95)) and float(opt.grad_norm) == 0.0
        assert all((x == 0).all() for x in opt.moments(0)) and int(opt.steps) == 1


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3e38])
def test_a_norm_that_is_not_finite_changes_nothing(value, bits):
    opt, grads, decays = group(4, [300, 70000, 5], KINDS["mixed"], bits, 1.0)
    opt.step(grads())
    before = [p.clone() for p in opt.params] + [getattr(opt, n).clone().reshape(-1).view(torch.uint8) for n in opt._STATE
                                                if getattr(opt, n) is not None]
    bad = grads()
    bad[1][69999] = value
    opt.step(bad)
    after = list(opt.params) + [getattr(opt, n).reshape(-1).view(torch.uint8) for n in opt._STATE if getattr(opt, n) is not None]
    assert all(torch.equal(a, b) for a, b in zip(after, before)) and not torch.isfinite(opt.grad_norm).all()
    check_step(opt, grads(), decays, 1.0)  # and the next one counts on


def test_past_32_bits_of_elements():
    """A tensor of more than 2^31 elements: its ends, in 8 bits."""
    from shifted_window_attention_cyclic_gb300.optim import AdamW, grad_norm
    n = 2**31 + 777
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 2**31 - 1, 2**31, n - 2, n - 1], device="cuda")
    g[at] = torch.tensor([1.0, -2.0, 3.0, -4.0, 5.0, -6.0], device="cuda").bfloat16()
    assert abs(float(grad_norm([g])) - 91**0.5) <= 1e-5
    opt = AdamW([p], lr=0.5, state_bits=8, max_norm=100.0)
    opt.step([g])
    assert abs(float(opt.grad_norm) - 91**0.5) <= 1e-5
    assert torch.allclose(p[at], -0.5 * torch.sign(g[at].float()), rtol=1e-4) and int((p != 0).sum()) == 6
    m, _ = opt.moments(0)
    assert (m[at] != 0).all() and int((opt.m.view(torch.uint8) != 0).sum()) == 6


@pytest.mark.parametrize("kinds", [[F], [B], [F, B]])
def test_norm(kinds):
    from shifted_window_attention_cyclic_gb300.optim import grad_norm
    gen = torch.Generator().manual_seed(5)
    for sizes, off in (([1], 0), (SIZES, 0), (SIZES, 3), ([3_000_017, 12], 1), ([50] * 2100, 0), ([0], 0)):
        ts = [tensor(gen, n, kinds[i % len(kinds)], 1.0 + i % 3, off, 0.2) for i, n in enumerate(sizes)]
        want = torch.sqrt(sum((t.double() ** 2).sum() for t in ts)).cpu().view(1)
        got = grad_norm(ts)
        assert got.shape == () and torch.equal(got, grad_norm(ts, out=torch.zeros((), device="cuda")))
        near("norm", got, want, NORM * want)


def test_clipping_factor():
    """A norm below the bound leaves gradients as they are, one above it scales them onto it."""
    from shifted_window_attention_cyclic_gb300.optim import AdamW
    g = torch.tensor([3.0, 4.0], device="cuda")
    for bound, factor in ((5.0, 1.0), (10.0, 1.0), (2.5, 0.5)):
        p = torch.zeros(2, device="cuda")
        opt = AdamW([p], betas=(0.5, 0.5), max_norm=bound)
        opt.step([g])
        assert float(opt.grad_norm) == 5.0 and torch.equal(opt.moments(0)[0], 0.5 * factor * g)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps(bits):
    """Every replay counts a step and reads the learning rate that it finds; same bits as steps one by one."""
    opt, grads, _ = group(6, [1000, 30000, 64], KINDS["mixed"], bits, 1.0)
    other, _, _ = group(6, [1000, 30000, 64], KINDS["mixed"], bits, 1.0)
    g = grads()
    opt.step(g), other.step(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(g)
    assert int(opt.steps) == 1
    for k in range(3):
        for o in (opt, other):
            o.lr.fill_(0.01 / (k + 1))
        graph.replay()
        other.step(g)
    torch.cuda.synchronize()
    assert int(opt.steps) == int(other.steps) == 4
    assert all(torch.equal(a, b) for a, b in zip(opt.params, other.params))
    assert torch.equal(opt.m.view(torch.uint8), other.m.view(torch.uint8)) and torch.equal(opt.grad_norm, other.grad_norm)


def test_parameters_of_autograd():
    from shifted_window_attention_cyclic_gb300.optim import AdamW
    w = torch.randn(8, 8, device="cuda", requires_grad=True)
    idle = torch.randn(5, device="cuda", requires_grad=True)
    opt, was = AdamW([w, idle], lr=0.1), idle.detach().clone()
    x = torch.randn(8, 8, device="cuda", requires_grad=True)
    y = x * w  # (a matrix product would leave its library's workspace in the allocator, which later tests count)
    y.sum().backward(retain_graph=True)
    opt.step()
    assert torch.equal(idle.detach(), was) and w.requires_grad
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()  # w is not what the forward saved
    opt.zero_grad()
    assert w.grad is None
    opt.step()  # nothing to do
    assert int(opt.steps) == 1


def test_state_dict():
    for bits in (32, 8):
        opt, grads, _ = group(7, SIZES, KINDS["mixed"], bits, 1.0)
        for _ in range(2):
            opt.step(grads())
        other, _, _ = group(7, SIZES, KINDS["mixed"], bits, 1.0)
        state = opt.state_dict()
        other.load_state_dict(state)
        with torch.no_grad():
            for p, q in zip(other.params, opt.params):
                p.copy_(q)
        g = grads()
        opt.step(g), other.step(g)
        assert all(torch.equal(a, b) for a, b in zip(opt.params, other.params)) and int(other.steps) == 3
        bad, _, _ = group(7, SIZES[1:], KINDS["mixed"], bits)
        with pytest.raises(ValueError):
            bad.load_state_dict(state)
        with pytest.raises(ValueError):
            other.load_state_dict({**state, "state_bits": 40 - bits})


def test_refusals_on_the_device():
    from shifted_window_attention_cyclic_gb300.optim import AdamW, grad_norm
    p = torch.zeros(64, device="cuda")
    opt = AdamW([p])
    for g in ([], [p.double()], [p[:32]], [torch.zeros(64, 2, device="cuda")[:, 0]], [torch.zeros(64)], [1.0]):
        with pytest.raises(ValueError):
            opt.step(g)
    for ps in ([p, p], [p, p[32:]], [torch.zeros(4, 4, device="cuda").t()], [p.half()]):
        with pytest.raises(ValueError):
            AdamW(ps)
    with pytest.raises(Exception):
        opt.step([p])  # a gradient over its parameter
    for name in ("lr", "steps", "m", "v"):  # another tensor in the place of one whose address the calls take
        with pytest.raises(AttributeError):
            setattr(opt, name, 0.1)
    with pytest.raises(ValueError):
        grad_norm([p], out=torch.zeros(2, device="cuda"))
    p.data = torch.zeros(32, device="cuda")
    with pytest.raises(ValueError):
        opt.step([torch.zeros(64, device="cuda")])
    assert int(opt.steps) == 0
