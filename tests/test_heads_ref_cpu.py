"""The 64-bit reference of the heads against what defines it: central
differences, rotations that compose; and the frequencies of Rotary."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import heads_ref as ref  # noqa: E402

STEP = 1e-5  # central differences of smooth functions in 64 bits: off by STEP^2 and 1e-16 / STEP


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
def test_gradient_against_differences(kind, layout):
    gen = torch.Generator().manual_seed(3)
    x, dy, d = (torch.randn(2, 3, 2, 32, generator=gen, dtype=torch.float64) for _ in range(3))
    some = kind != "none"
    gamma = torch.randn(32, generator=gen, dtype=torch.float64) + 1 if some else None
    beta = torch.randn(32, generator=gen, dtype=torch.float64) if some else None
    t = ref.turns(ref.grid_positions(2, (3,)) * 7, [0.9**j for j in range(8)], [0] * 8)
    (dx, dgamma, dbeta), _ = ref.heads_bwd(x, dy, t, layout, 1.3, kind, 1e-5, gamma)

    def loss(x, gamma, beta):
        return (ref.heads_fwd(x, t, layout, 1.3, kind, 1e-5, gamma, beta)[0] * dy).sum()

    got = (loss(x + STEP * d, gamma, beta) - loss(x - STEP * d, gamma, beta)) / (2 * STEP)
    assert abs(got - (dx * d).sum()) <= 1e-8 * (dx * d).abs().sum()
    if some:
        e = torch.randn(32, generator=gen, dtype=torch.float64)
        got = (loss(x, gamma + STEP * e, beta) - loss(x, gamma - STEP * e, beta)) / (2 * STEP)
        assert abs(got - (dgamma * e).sum()) <= 1e-8 * (dgamma * e).abs().sum()
        got = (loss(x, gamma, beta + STEP * e) - loss(x, gamma, beta - STEP * e)) / (2 * STEP)
        assert abs(got - (dbeta * e).sum()) <= 1e-8 * (dbeta * e).abs().sum()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scores_depend_on_the_distance_alone(layout):
    """What rotary positions are for: q at i and k at j meet as at i + n and j + n."""
    gen = torch.Generator().manual_seed(4)
    q, k = (torch.randn(1, 1, 1, 32, generator=gen, dtype=torch.float64) for _ in range(2))
    freq = [10000.0 ** (-j / 16) for j in range(16)]

    def score(i, j):
        at = lambda p: ref.turns(torch.tensor([[[p]]]), freq, [0] * 16)  # noqa: E731
        return (ref.rotate(q, at(i), layout)[0] * ref.rotate(k, at(j), layout)[0]).sum()

    for i, j in ((0, 0), (5, 2), (-3, 11)):
        for n in (1, 1000, 123456789012):
            assert abs(score(i, j) - score(i + n, j + n)) <= 1e-12


def test_rotary_frequencies():
    from shifted_window_attention_cyclic_gb300.heads import Rotary
    r = Rotary(32, base=10000.0)
    assert r.frequencies == [10000.0 ** (-j / 16) for j in range(16)] and r.amplitude == 1.0
    r = Rotary(32, axes=3)
    assert [r.axis_of.count(a) for a in range(3)] == [5, 5, 6] and r.frequencies[:5] == [10000.0 ** (-j / 5) for j in range(5)]
    linear, ntk = (Rotary(64, scaling=s, factor=8.0) for s in ("linear", "ntk"))
    plain = Rotary(64)
    assert linear.frequencies == [f / 8 for f in plain.frequencies]
    assert ntk.frequencies[0] == 1.0 and math.isclose(ntk.frequencies[-1], plain.frequencies[-1] / 8, rel_tol=1e-12)
    yarn = Rotary(64, scaling="yarn", factor=8.0, trained=1000)
    for f, g in zip(plain.frequencies, yarn.frequencies):
        n = 1000 * f / (2 * math.pi)
        assert g == f if n >= 32 else math.isclose(g, f / 8) if n <= 1 else f / 8 < g < f
    assert math.isclose(yarn.amplitude, 0.1 * math.log(8) + 1)
    # fixed point: half a unit of 2^-64 turns from the frequency
    for r in (plain, yarn):
        for f, k in zip(r.frequencies, r._freq):
            assert abs(ref.Fraction(f) / (2 * ref.PI) - ref.Fraction(int(k), 2**64)) <= ref.Fraction(1, 2**65)
    wide = Rotary(16, frequencies=[-0.5] + [7.0] * 7)  # any sign, more than a turn
    assert abs(ref.Fraction(-0.5) / (2 * ref.PI) + 1 - ref.Fraction(int(wide._freq[0]), 2**64)) <= ref.Fraction(1, 2**65)
    assert abs(ref.Fraction(7.0) / (2 * ref.PI) - 1 - ref.Fraction(int(wide._freq[1]), 2**64)) <= ref.Fraction(1, 2**65)
