"""Window attention with dropped probabilities on the GPU where one bar for a
whole tensor says nothing: the dBias of head_dim 128 whose delta comes from the
given O, and rates that drop nearly every pair."""
import pytest

torch = pytest.importorskip("torch")

from tests.attn_dropout_bars import Pairs, over  # noqa: E402
from tests.parity_util import BF16_MAX_ABS, BF16_REL_L2  # noqa: E402
from tests.test_gpu_attn_dropout import CASES, LARGE, run  # noqa: E402

pytestmark = pytest.mark.gpu

KEY = (2**64 - 3, 9)  # seed and step of run()
GIVEN_O = LARGE[:4]
# with sites at which some visible pairs are kept
EXTREME = [(CASES[0], 290), (CASES[4], 1), (CASES[7], 44), (LARGE[2], 14)]


@pytest.mark.parametrize("case", GIVEN_O, ids=lambda c: "x".join(map(str, c[0])))
def test_dbias_of_a_given_o(case):
    """Within six standard deviations of what the roundings of O and P leave in each bias row, beside the bar of every
    max-abs comparison, and within the relative bar of dBias elsewhere."""
    _, _, got, _ = run(case, 0.3, give_o=True)
    pr = Pairs(case, 0.3, *KEY, 6)
    g, want = got["dbias"].double().cpu(), pr.rows(pr.ds())
    assert over(g, want, 6 * pr.dbias_deviation() + BF16_MAX_ABS * pr.c) <= 0
    assert (g - want).norm() <= BF16_REL_L2 * want.norm()


@pytest.mark.parametrize("case,site", EXTREME, ids=["simt", "one_window", "two_windows", "large"])
def test_the_few_kept_pairs_at_an_extreme_rate(case, site):
    rate = 65535 / 65536
    _, _, got, _ = run(case, rate, site=site)
    pr = Pairs(case, rate, *KEY, site)
    want, bound = pr.outputs(), pr.bounds()
    for name in want:
        g = got[name].double().cpu().view(want[name].shape)
        assert over(g, want[name], bound[name]) <= 0, name
