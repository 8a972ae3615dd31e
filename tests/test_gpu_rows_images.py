"""Rows cut into images in several ways: the norm, and a join without gate and
path, do not look at images, neither in their results nor in their memory."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_rows import ALL, join_case  # noqa: E402

pytestmark = pytest.mark.gpu

UNGATED = tuple(n for n in ALL if n != "gate")


def grown(call):
    """What `call` returns, and the most memory it held beside what was there."""
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = call()
    return out, torch.cuda.max_memory_allocated() - before


@pytest.mark.parametrize("shape", [(4608,), (48, 96), (2, 48, 48)], ids=str)
@pytest.mark.parametrize("channels,dtype", [(64, "bf16"), (256, "bf16"), (384, "f32"), (1032, "bf16")])
def test_any_cut_gives_the_same_bits_in_the_same_memory(channels, dtype, shape):
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    case, par, _, drop, _, _, _ = join_case(channels, 1, 4608, channels, dtype, "layer", "rms", UNGATED, 0.2, 0.0)
    x, z, dy, dh = (case[n][0] for n in ("x", "z", "dy", "dh"))
    norm, join = BlockNorm(channels, "layer", dtype=dtype), ResidualJoin(channels, "layer", "rms", dtype=dtype)
    got = []
    for cut in ((1, 4608), shape):
        a, b, da, db = (t.view(*cut, channels) for t in (x, z, dy, dh))
        y, h = join.forward(a, b, **par, drop=drop)
        n, held_n = grown(lambda: norm.backward(a, da, par["pre_gamma"], par["pre_beta"]))
        j, held_j = grown(lambda: join.backward(y, b, da, db, **par, drop=drop))
        got.append(((norm.forward(a), y, h) + n + tuple(t for t in j if t is not None), held_n, held_j))
    assert len(got[0][0]) == 13
    assert all(torch.equal(p.flatten(), q.flatten()) for p, q in zip(got[0][0], got[1][0]))
    assert got[1][1] <= got[0][1] and got[1][2] <= got[0][2]


def test_workspace_without_a_gate_does_not_grow_with_the_images():
    """1 179 648 rows of 64 channels as images of one row: a slot of two column sums for each image would be 604 MB."""
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
    x = torch.ones(1179648, 64, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(64, device="cuda")
    for call, outputs in ((lambda: BlockNorm(64).backward(x, x, g, g), 1),
                          (lambda: ResidualJoin(64, "none", "layer").backward(x, x, x, x, pre_gamma=g, scale=g), 2)):
        assert grown(call)[1] <= outputs * x.numel() * 2 + (4 << 20)
    # the library's own calls ask for no more than one image's workspace either
    rows, one = C.swin_attn_rows(1179648, 1, 64, C.SWIN_BF16), C.swin_attn_rows(1, 1179648, 64, C.SWIN_BF16)
    ws = torch.empty(C.swin_attn_rows_workspace_bytes(one), dtype=torch.uint8, device="cuda")
    dx, dz, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(g)
    norm, none, off = C.swin_attn_norm(C.SWIN_NORM_LAYER, 1e-5, None, None), C.swin_attn_norm(0, 1e-5, None, None), C.swin_attn_drop(0.0, 0, None)
    C.swin_attn_norm_bwd(rows, x, norm, x, None, dx, dg, None, ws)
    join = C.swin_attn_join(none, norm, g.data_ptr(), None, off, off)
    grads = C.swin_attn_join_grads(None, None, dg.data_ptr(), None, None, None)
    C.swin_attn_join_bwd(rows, x, x, join, x, x, dx, dz, grads, ws)
    # a gate's gradient needs its slots
    gate = torch.ones(1179648, 64, device="cuda")
    join = C.swin_attn_join(none, norm, None, gate.data_ptr(), off, off)
    with pytest.raises(C.SwinAttnError, match=r"\(%d\)" % C.SWIN_ERR_WORKSPACE):  # (kept, it would keep the tensors)
        C.swin_attn_join_bwd(rows, x, x, join, x, x, dx, dz, grads, ws)
    torch.cuda.synchronize()


def test_gates_of_images_without_rows():
    """Images that hold no tokens have gradients of zero, and take no workspace for what they do not sum."""
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    x, gate = torch.empty(300000, 0, 64, device="cuda"), torch.ones(300000, 64, device="cuda")
    assert C.swin_attn_rows_workspace_bytes(C.swin_attn_rows(300000, 0, 64, C.SWIN_F32)) <= 2 << 20
    out = ResidualJoin(64, dtype="f32").backward(x, x, x, gate=gate)
    assert out.dgate.shape == gate.shape and not out.dgate.any()
