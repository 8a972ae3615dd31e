"""The 64-bit references themselves: the generator against published answers,
the decisions' share, and every written-out gradient against central
differences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import rows_ref as ref  # noqa: E402


@pytest.mark.parametrize("rounds,ctr,key,want", [
    (7, (0, 0, 0, 0), 0, "5f6fb709 0d893f64 4f121f81 4f730a48"),
    (10, (0, 0, 0, 0), 0, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    (10, (0xffffffff,) * 4, 2**64 - 1, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    (10, (0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), 0x299f31d0a4093822,
     "d16cfe09 94fdcceb 5001e420 24126ea1"),
])
def test_generator_known_answers(rounds, ctr, key, want):
    got = ref.philox4x32(*[np.uint64(c) for c in ctr], key, rounds)
    assert " ".join("%08x" % int(w) for w in got) == want


def test_decisions_share_and_independence():
    n = 1 << 18
    for rate in (0.1, 0.5):
        k = ref.keep(np.arange(n), 1234567, 3, 5, rate)
        # six standard deviations of a binomial share
        assert abs(k.mean() - (1 - ref.threshold(rate) / 65536)) < 6 * np.sqrt(rate * (1 - rate) / n)
        for other in (ref.keep(np.arange(n), 1234567, 4, 5, rate), ref.keep(np.arange(n), 1234567, 3, 6, rate),
                      ref.keep(np.arange(n), 1234568, 3, 5, rate), np.roll(k, 1)):
            agree = (k == other).mean()
            want = (1 - rate) ** 2 + rate**2
            assert abs(agree - want) < 6 * np.sqrt(want * (1 - want) / n)


def _num(f, t):
    """Gradient of the number f() by central differences in every element of t (float64)."""
    g = torch.zeros_like(t)
    flat, out = t.view(-1), g.view(-1)
    for i in range(flat.numel()):
        x = flat[i].item()
        flat[i] = x + 1e-6
        hi = f()
        flat[i] = x - 1e-6
        lo = f()
        flat[i] = x
        out[i] = (hi - lo) / 2e-6
    return g


@pytest.mark.parametrize("post,pre", [("none", "layer"), ("layer", "rms"), ("rms", "none"), ("rms", "layer")])
def test_join_gradients_against_differences(post, pre):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    b, t, c = 2, 3, 8
    x, z, dy, dh = r(b, t, c), r(b, t, c), r(b, t, c), r(b, t, c)
    par = {k: r(c) for k in ("scale", "post_gamma", "post_beta", "pre_gamma", "pre_beta")}
    par["gate"] = r(b, c)
    if post == "none":
        del par["post_gamma"], par["post_beta"]
    if pre == "none":
        del par["pre_gamma"], par["pre_beta"]
    drop, path = (7, 1, 2, 0.3), (7, 1, 3, 0.4)

    def loss():
        y, h = ref.join_fwd(x, z, post, pre, 1e-5, par, drop, path)
        return float((y * dy).sum() + (0.0 if h is None else (h * dh).sum()))

    y, _ = ref.join_fwd(x, z, post, pre, 1e-5, par, drop, path)
    grad, size = ref.join_bwd(y, z, dy, None if pre == "none" else dh, post, pre, 1e-5, par, drop, path)
    for name, t_ in [("dx", x), ("dz", z)] + [("d" + k, v) for k, v in par.items()]:
        assert torch.allclose(grad[name], _num(loss, t_), atol=1e-6, rtol=1e-6), name
        assert (size[name] >= grad[name].abs() - 1e-12).all(), name


def test_attention_gradients_against_differences():
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    # two windows of 4 slots over 7 tokens (one pad), two regions in the first
    src = np.array([[0, 1, 2, 3], [4, 5, 6, -1]])
    region = np.array([[0, 0, 1, 1], [0, 0, 0, 0]])
    rel = np.arange(4)[:, None] - np.arange(4)[None] + 3
    heads, hd = 2, 4
    q, k, v, dout = (r(1, 7, heads * hd) for _ in range(4))
    bias = r(7, heads)
    land = torch.zeros((1, 7), dtype=torch.bool)
    land[0, 5] = True
    args = dict(land=land, tables=(src, region, rel), heads=heads, drop=(9, 1, 2, 0.3))
    got = ref.attn(q, k, v, bias, dout=dout, **args)

    def loss():
        return float((ref.attn(q, k, v, bias, **args)["o"] * dout).sum())

    for name, t in (("dq", q), ("dk", k), ("dv", v), ("dbias", bias)):
        assert torch.allclose(got[name], _num(loss, t), atol=1e-6, rtol=1e-6), name
