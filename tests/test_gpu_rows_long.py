"""Norm, join and dropout at sizes whose offsets pass 32 bits and whose column
sums are long, against float64 on the same GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import rows_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

E32 = 2.0**-24


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 2**30:
        pytest.skip("needs %d GB" % gigabytes)


def test_dropout_of_more_than_2_to_35_elements():
    """The generator's block number passes 32 bits, and so does every division by a span."""
    room(80)
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, apply_dropout
    n, site = 2**35 + 83, 3
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    state = DropoutState(77, 2)
    for span, rate in ((1, 0.5), (2**20 + 8, 0.5), (3, 0.5)):
        x.fill_(1.0)
        apply_dropout(x, Dropout(state, rate, site), span, out=x)
        for a in (0, 2**31 - 40, 2**32 - 40, 2**32 + 8 * (2**20 + 8) - 40, 3 * 2**33 - 40, 2**35 - 40, n - 83):
            got = x[a:a + 83].float().cpu().numpy()
            keep = ref.keep(np.arange(a, a + 83, dtype=np.uint64) // np.uint64(span), 77, 2, site, rate)
            assert np.array_equal(got, np.where(keep, 2.0, 0.0)), (span, a)
        del got
    del x
    torch.cuda.empty_cache()


def test_rows_past_2_to_32_elements():
    """Rows behind 2^32 elements (8 GB): the norm's are those of the same rows alone, the join's drop by their own place."""
    room(70)
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    t, c = 524288 + 1003, 8192
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randn(1, 7, c, generator=gen, device="cuda").bfloat16()
    gamma = torch.randn(c, generator=gen, device="cuda")
    x = torch.ones(1, t, c, dtype=torch.bfloat16, device="cuda")
    x[:, -7:] = last
    norm = BlockNorm(c, "rms")
    h = norm.forward(x, gamma)
    assert torch.equal(h[:, -7:], norm.forward(last, gamma)) and torch.equal(h[:, :5], norm.forward(x[:, :5], gamma))
    dx = norm.backward(x, x, gamma, dx=h, want_params=False)[0]
    assert torch.equal(dx[:, -7:], norm.backward(last, last, gamma, want_params=False)[0])
    del h, dx
    drop = Dropout(DropoutState(5), 0.5, 9)
    index = np.arange((t - 7) * c, t * c, dtype=np.uint64)
    assert index[0] > 2**32
    keep = torch.from_numpy(ref.keep(index, 5, 0, 9, 0.5)).view(1, 7, c).cuda()
    join = ResidualJoin(c)
    y, _ = join.forward(x, x, drop=drop)
    assert torch.equal(y[:, -7:], torch.where(keep, last.float() * 3, last.float()).bfloat16())
    del y
    out = join.backward(x, x, x, drop=drop, want_params=False)
    assert torch.equal(out.dx[:, -7:], last) and torch.equal(out.dz[:, -7:], torch.where(keep, 2 * last, 0 * last))
    del out, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,channels,dtype", [(1179648, 64, "bf16"), (300001, 1024, "bf16"), (100003, 4096, "f32"),
                                                 (50021, 8192, "f32")])
def test_long_column_sums(rows, channels, dtype):
    """A bias of the sums would grow with their length: terms of one sign (mean 1), hundreds to thousands a thread. An
    fp32 sum is off by at most one rounding an addition: those of a thread (the rows over one CTA an SM at the least)
    and of the fold; xhat by the 96 roundings of a row."""
    room(40)
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    gen = torch.Generator(device="cuda").manual_seed(channels)
    tdt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x, dh = ((torch.randn(1, rows, channels, generator=gen, device="cuda") * s + m).to(tdt) for s, m in ((1.0, 0.5), (0.5, 1.0)))
    g = torch.rand(channels, generator=gen, device="cuda") + 0.5
    gate = torch.rand(1, channels, generator=gen, device="cuda") + 0.5
    longest = (rows / 152 + 64) * E32
    _, dgamma, dbeta = BlockNorm(channels, "rms", dtype=dtype).backward(x, dh, g, g)
    out = ResidualJoin(channels, dtype=dtype).backward(x, x, dh, scale=g, gate=gate)
    sums = {k: torch.zeros(channels, dtype=torch.float64, device="cuda") for k in ("hat", "hat_abs", "dh", "dh_abs", "z", "z_abs")}
    for a in range(0, rows, 16384):
        u, v = x[0, a:a + 16384].double(), dh[0, a:a + 16384].double()
        hat = u / torch.sqrt(u.square().mean(-1, keepdim=True) + 1e-5)
        for k, term in (("hat", v * hat), ("dh", v), ("z", v * u)):
            sums[k] += term.sum(0)
            sums[k + "_abs"] += term.abs().sum(0)
    g64, gate64 = g.double(), gate[0].double()

    def close(got, want, size, relative):
        assert ((got.double().flatten() - want).abs() <= relative * size).all()

    close(dgamma, sums["hat"], sums["hat_abs"], longest + 96 * E32)
    close(dbeta, sums["dh"], sums["dh_abs"], longest)
    close(out.dscale, sums["z"] * gate64, sums["z_abs"] * gate64, longest + 8 * E32)
    close(out.dgate, sums["z"] * g64, sums["z_abs"] * g64, longest + 8 * E32)
