"""Window attention with dropped probabilities on the GPU, against the 64-bit
reference that draws the decisions by itself. The bars are those of the
attention without dropout, times the kept scale that multiplies every term of
O, dQ, dK, dV and dBias."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import workloads  # noqa: E402
from tests import rows_ref as ref  # noqa: E402
from tests.parity_util import BF16_MAX_ABS, BF16_REL_L2, F32_MAX_ABS, errors, host, to_device  # noqa: E402

pytestmark = pytest.mark.gpu

# grid, window, shift, periodic, heads, head_dim, batch, dtype, land: one and two windows per tile, ragged and
# wrapping windows, pads, a window of one slot and of 128, odd slot counts, land, the SIMT kernels in both types
CASES = [
    ((16, 32), (4, 8), (2, 4), (0, 0), 2, 16, 1, "f32", None),
    ((9, 13), (4, 4), (2, 2), (0, 1), 3, 32, 2, "f32", (0.4, 0.4)),
    ((7, 11), (3, 5), (1, 2), (1, 0), 2, 16, 1, "bf16", None),
    ((24, 36), (6, 12), (3, 6), (0, 1), 4, 32, 2, "bf16", None),
    ((21, 30), (8, 8), (4, 4), (0, 1), 3, 32, 1, "bf16", (0.3, 0.3)),
    ((20, 27), (8, 12), (4, 6), (0, 1), 2, 32, 1, "bf16", (0.3, 0.3)),
    ((4, 17, 24), (2, 8, 8), (1, 4, 4), (0, 0, 1), 2, 32, 1, "bf16", (0.3, 0.6)),
    ((10, 14), (5, 7), (2, 3), (1, 1), 3, 32, 2, "bf16", None),
    ((6, 9), (1, 1), (0, 0), (0, 0), 2, 32, 1, "bf16", None),
    ((5, 130), (1, 128), (0, 64), (0, 1), 1, 32, 1, "bf16", None),
    ((1, 1), (2, 3), (0, 0), (0, 0), 1, 32, 1, "bf16", None),
    ((30, 41), (3, 3), (1, 1), (0, 1), 5, 32, 1, "bf16", (1.0, 1.0)),
]


# head_dim 128, windows of any size: one partial key tile, two tiles, a partial second one, ragged 3-D with land,
# more than one image, windows above 2 048 slots (without a bias: two query stages), 32 key tiles (slots in runs)
LARGE = [
    ((21, 45), (8, 12), (4, 6), (0, 1), 2, 128, 2, "bf16", None),
    ((32, 40), (16, 16), (8, 8), (0, 1), 2, 128, 1, "bf16", (0.3, 0.3)),
    ((14, 27), (12, 12), (6, 6), (1, 0), 1, 128, 2, "bf16", None),
    ((3, 40, 70), (2, 16, 16), (1, 8, 8), (0, 0, 1), 1, 128, 1, "bf16", (0.2, 0.5)),
    ((60, 100), (30, 100), (15, 50), (0, 1), 1, 128, 1, "bf16", None),
    ((64, 72), (64, 64), (32, 32), (0, 1), 1, 128, 1, "bf16", None),
]


def run(case, rate, site=6, seed_index=700, want_bias=True, give_o=False):
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
    grid, window, shift, periodic, heads, hd, batch, dtype, land_p = case
    wl = workloads.custom(grid, window, shift, periodic, heads, hd, batch, dtype, land_p, seed_index=seed_index)
    x = workloads.generate(wl)
    attn = SwinWindowAttention(grid, window, shift, periodic, heads, hd, batch, dtype, wl.has_land)
    t = to_device(x, wl, torch.device("cuda", 0))
    bias = t["bias"] if want_bias else None
    drop = Dropout(DropoutState(2**64 - 3, 9), rate, site)
    o, lse = attn.forward(t["q"], t["k"], t["v"], bias, t["land"], dropout=drop)
    dq, dk, dv, dbias = attn.backward(t["q"], t["k"], t["v"], t["dout"], lse, bias, t["land"], dropout=drop,
                                      o=o if give_o else None, want_dbias=want_bias or hd != 128)
    torch.cuda.synchronize()
    assert C.swin_attn_status(attn.plan) == 0
    got = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv, dbias=dbias)
    tables = C.swin_attn_plan_tables(attn.plan)
    flat = lambda n: torch.from_numpy(x[n]).double().reshape(batch, -1, heads * hd)  # noqa: E731
    land = None if x["land"] is None else torch.from_numpy(x["land"]).reshape(batch, -1) != 0
    b64 = torch.from_numpy(x["bias"]).double()
    rel = tables[3]
    if rel is None:  # a plan keeps the slot pairs' bias rows up to 2 048 slots; without a bias any row will do
        assert not want_bias
        rel = np.zeros((tables[0].shape[1],) * 2, np.int64)
    want = ref.attn(flat("q"), flat("k"), flat("v"), b64 if want_bias else 0 * b64, land, (tables[0], tables[1], rel), heads,
                    (2**64 - 3, 9, site, rate), flat("dout"))
    return attn, t, got, want


@pytest.mark.parametrize("rate", [0.1, 0.5])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[0])) + "_" + c[7])
def test_parity(case, rate):
    _, _, got, want = run(case, rate)
    c = ref.kept_scale(rate)
    for n in ("o", "dq", "dk", "dv", "dbias"):
        max_abs, rel = errors(host(got[n]).reshape(want[n].shape), want[n].numpy())
        if case[7] == "f32":
            assert max_abs <= F32_MAX_ABS * c, (n, max_abs)
        else:
            # windows of one slot: dS = P (dP - P dP) with P = 1 is 0, and a relative error has no meaning
            # (P is off by a few 2^-23 of the exponential, so dQ and dK by that times |dP| |k|: the max-abs bar holds it)
            zero = not want[n].any()
            assert max_abs <= BF16_MAX_ABS * c and (zero or rel <= BF16_REL_L2), (n, max_abs, rel)
    lse = host(got["lse"]).reshape(want["lse"].shape)
    sea = np.isfinite(want["lse"].numpy())
    assert (lse[~sea] == -np.inf).all() and np.abs(lse[sea] - want["lse"].numpy()[sea]).max(initial=0) <= 1e-4


@pytest.mark.parametrize("give_o", [False, True], ids=["delta_summed", "delta_from_o"])
@pytest.mark.parametrize("case", LARGE, ids=lambda c: "x".join(map(str, c[0])))
def test_parity_large(case, give_o):
    n = int(np.prod(case[1]))
    want_bias = n <= 2048
    rate = 0.3 if give_o else 0.1
    _, _, got, want = run(case, rate, want_bias=want_bias, give_o=give_o)
    c = ref.kept_scale(rate)
    for name in ("o", "dq", "dk", "dv") + (("dbias",) if want_bias and not give_o else ()):
        max_abs, rel = errors(host(got[name]).reshape(want[name].shape), want[name].numpy())
        assert max_abs <= BF16_MAX_ABS * c and rel <= BF16_REL_L2, (name, max_abs, rel)
    if want_bias and give_o:
        # delta = dO . O carries O's rounding, half a step of 2^-8 |O|: a row's dS is off by P times
        # sum_c |dO_c| 2^-9 |O_c| at most, and a bias row adds up its pairs' errors
        d = torch.from_numpy(workloads.generate(workloads.custom(*case[:9], seed_index=700))["dout"]).double()
        heads = case[4]
        slack = (d.reshape(case[6], -1, heads, 128).abs() * want["o"].view(case[6], -1, heads, 128).abs()).sum(-1) * 2.0**-8
        assert np.abs(host(got["dbias"]) - want["dbias"].numpy()).max() <= BF16_MAX_ABS * c + float(slack.sum((0, 1)).max())
    lse = host(got["lse"]).reshape(want["lse"].shape)
    sea = np.isfinite(want["lse"].numpy())
    # the bar of the large windows' log-sum-exp (lazy rescaling sums P in another order)
    assert (lse[~sea] == -np.inf).all() and np.abs(lse[sea] - want["lse"].numpy()[sea]).max(initial=0) <= 2e-3


@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[7], LARGE[2]],
                         ids=["simt", "one_window", "two_windows", "large"])
def test_every_key_of_a_row_dropped(case):
    """At a rate of 65535/65536 nearly every decision drops: O is 0 there, not NaN, and what is kept is scaled by 65536."""
    _, _, got, want = run(case, 65535 / 65536)
    for n in ("o", "dq", "dk", "dv", "dbias"):
        g, w = host(got[n]).reshape(want[n].shape), want[n].numpy()
        assert np.isfinite(g).all()
        # rounding is relative to the kept terms, each of the size of 65536 P V
        assert np.abs(g - w).max() <= (2e-2 if case[7] == "bf16" else 1e-5) * 65536
        if n in ("o", "dv"):
            assert (g[w == 0] == 0).all()


def test_simt_and_tensor_core_kernels_drop_the_same():
    """One plan geometry on both kernel families (bf16, head_dim 32): the same keys are dropped, so V = one-hot rows
    read the same zeros out of P."""
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
    drop = Dropout(DropoutState(41), 0.4, 2)
    got = []
    for impl in ("simt", "tc"):
        attn = SwinWindowAttention((8, 12), (4, 8), (2, 4), (0, 1), 2, 32, 2, "bf16", impl=impl)
        gen = torch.Generator().manual_seed(1)
        q, k = (torch.randn(attn.shape, generator=gen).bfloat16().cuda() for _ in range(2))
        # token (r, c) has a one in channel 8 (r % 4) + c % 8: another channel for every token of a window
        ch = 8 * (torch.arange(8)[:, None] % 4) + torch.arange(12) % 8
        v = torch.nn.functional.one_hot(ch, 32).bfloat16()[None, :, :, None].expand(2, 8, 12, 2, 32)
        got.append(attn.forward(q, k, v.reshape(attn.shape).contiguous().cuda(), dropout=drop)[0])
    assert torch.equal(got[0] == 0, got[1] == 0) and 0.3 < (got[0] == 0).float().mean() < 0.95
    assert (got[0].float() - got[1].float()).abs().max() <= BF16_MAX_ABS * ref.kept_scale(0.4)


def test_block_pair_takes_a_dropout_for_each_layer():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinBlockPair
    pair = SwinBlockPair((16, 24), (4, 8), (0, 1), 2, 32)
    layers = [tuple(torch.randn(pair.wmsa.shape, device="cuda").bfloat16() for _ in range(3)) + (pair.wmsa.new_bias(),)
              for _ in range(2)]
    dout = torch.randn(pair.wmsa.shape, device="cuda").bfloat16()
    state = DropoutState(4)
    drops = Dropout(state, 0.2, 0), Dropout(state, 0.2, 1)
    (o1, l1), (o2, l2) = pair.forward(*layers, dropout=drops)
    g1, g2 = pair.backward(*layers, dout, dout, l1, l2, dropout=drops)
    for attn, layer, drop, o, lse, g in ((pair.wmsa, layers[0], drops[0], o1, l1, g1),
                                         (pair.swmsa, layers[1], drops[1], o2, l2, g2)):
        assert torch.equal(attn.forward(*layer, dropout=drop)[0], o)
        want = attn.backward(*layer[:3], dout, lse, layer[3], dropout=drop)
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    assert not torch.equal(o1, pair.forward(*layers)[0][0])


def test_rate_zero_is_the_attention_without_dropout():
    for case in (CASES[0], CASES[4]):
        attn, t, got, _ = run(case, 2.0**-18)  # rounds to T = 0
        o, lse = attn.forward(t["q"], t["k"], t["v"], t["bias"], t["land"])
        grads = attn.backward(t["q"], t["k"], t["v"], t["dout"], lse, t["bias"], t["land"])
        for a, b in zip((o, lse) + grads, (got[n] for n in ("o", "lse", "dq", "dk", "dv", "dbias"))):
            assert torch.equal(a, b)


def test_without_bias_and_same_bits_again():
    case = CASES[5]
    _, _, got, want = run(case, 0.2, want_bias=False)
    _, _, again, _ = run(case, 0.2, want_bias=False)
    for n in ("o", "dq", "dk", "dv", "dbias"):
        assert torch.equal(got[n], again[n])
        _, rel = errors(host(got[n]).reshape(want[n].shape), want[n].numpy())
        assert rel <= BF16_REL_L2, n


def test_captured_replay_takes_the_step_of_the_state():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    attn, t, _, _ = run(CASES[4], 0.2)
    state = DropoutState(11)
    drop = Dropout(state, 0.2, 1)
    want = []
    for _ in range(3):
        want.append([x.clone() for x in attn.forward(t["q"], t["k"], t["v"], t["bias"], t["land"], dropout=drop)])
        state.advance()
    state.tensor[1] -= 3
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = attn.forward(t["q"], t["k"], t["v"], t["bias"], t["land"], dropout=drop)
        state.advance()
    for k in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[k]))
    assert not torch.equal(want[0][0], want[1][0]) and torch.equal(want[0][1], want[1][1])


def test_refusals():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
    attn = SwinWindowAttention((16, 16), (16, 16), (8, 8), (0, 1), 1, 128)
    q = torch.zeros(attn.shape, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="Dropout"):
        attn.forward(q, q, q, dropout=0.1)
    with pytest.raises(ValueError, match="its state"):
        attn.forward(q, q, q, dropout=Dropout(DropoutState(1, device="cpu"), 0.1, 0))
    with pytest.raises(ValueError, match="dtype"):
        attn.forward(q.float(), q, q, dropout=Dropout(DropoutState(1), 0.1, 0))
