"""The bars of attn_dropout_bars.py catch what they are there for: mistakes
planted in the reference, on the CPU."""
import pytest

torch = pytest.importorskip("torch")

from tests import rows_ref as ref  # noqa: E402
from tests.attn_dropout_bars import Pairs, over  # noqa: E402
from tests.parity_util import BF16_MAX_ABS, BF16_REL_L2  # noqa: E402
from tests.test_gpu_attn_dropout_bars import EXTREME, GIVEN_O, KEY  # noqa: E402


@pytest.mark.parametrize("case", GIVEN_O, ids=lambda c: "x".join(map(str, c[0])))
def test_wrong_dbias_of_a_given_o_is_seen(case):
    pr = Pairs(case, 0.3, *KEY, 6)
    want, sigma = pr.rows(pr.ds()), pr.dbias_deviation()
    bound = 6 * sigma + BF16_MAX_ABS * pr.c
    # what the roundings leave is well inside the relative bar, which is that of dBias elsewhere
    assert sigma.norm() <= BF16_REL_L2 / 3 * want.norm()
    for wrong in (0 * want, -want, pr.rows(pr.ds(scale=1.0)), want * 1.02):
        assert (wrong - want).norm() > BF16_REL_L2 * want.norm()
    for wrong in (0 * want, -want, pr.rows(pr.ds(scale=1.0))):
        assert over(wrong, want, bound) > 0


@pytest.mark.parametrize("case,site", EXTREME)
def test_wrong_scales_of_the_few_kept_are_seen(case, site):
    rate = 65535 / 65536
    pr = Pairs(case, rate, *KEY, site)
    kept = int((pr.keep * pr.visible).sum())
    assert kept >= 2 and pr.c == 65536
    want, bound = pr.outputs(), pr.bounds()
    wrong = pr.outputs(scale=65536 * (0.95 if case[7] == "bf16" else 0.999))
    for name in want:
        # mostly zeros, which are to be exact
        assert want[name].any() and (want[name] == 0).double().mean() > 0.5, name
        assert ((bound[name] == 0) == (want[name] == 0)).all() or name in ("dq", "dk", "dbias")
        for bad in (0 * want[name], wrong[name], -want[name]):
            assert over(bad, want[name], bound[name]) > 0, name


def test_the_reference_is_the_one_of_the_other_tests():
    from tests.attn_dropout_bars import oracle, problem_of, workloads
    case = GIVEN_O[0]
    wl = workloads.custom(*case[:9], seed_index=700)
    x, tab = workloads.generate(wl), oracle.tables(problem_of(wl))
    flat = lambda n: torch.from_numpy(x[n]).double().reshape(case[6], -1, case[4] * case[5])  # noqa: E731
    other = ref.attn(flat("q"), flat("k"), flat("v"), torch.from_numpy(x["bias"]).double(), None, (tab[0], tab[1], tab[3]),
                     case[4], KEY + (6, 0.3), flat("dout"))
    mine = Pairs(case, 0.3, *KEY, 6).outputs()
    for name in mine:
        assert torch.allclose(mine[name], other[name].view(mine[name].shape), rtol=0, atol=1e-10), name
