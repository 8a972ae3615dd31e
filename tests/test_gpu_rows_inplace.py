"""Parameter gradients written over their parameters, through the C entry points."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_rows import ALL, join_case  # noqa: E402

pytestmark = pytest.mark.gpu


# one image, a few, more than a lane each, more than one group of images
@pytest.mark.parametrize("images,tokens", [(1, 3000), (3, 700), (90, 7), (600, 5)])
def test_join_gradients_over_their_parameters(images, tokens):
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    from shifted_window_attention_cyclic_gb300.residual import ResidualJoin
    c = 200
    case, par, _, drop, path, _, _ = join_case(images, images, tokens, c, "bf16", "layer", "rms", ALL, 0.2, 0.3)
    x, z, dy, dh = (case[n][0] for n in ("x", "z", "dy", "dh"))
    join = ResidualJoin(c, "layer", "rms")
    y, _ = join.forward(x, z, **par, drop=drop, path=path)
    want = join.backward(y, z, dy, dh, **par, drop=drop, path=path)
    rows = C.swin_attn_rows(images, tokens, c, C.SWIN_BF16)
    ws = torch.empty(C.swin_attn_rows_workspace_bytes(rows), dtype=torch.uint8, device="cuda")
    p = {n: t.clone() for n, t in par.items()}
    at = {n: t.data_ptr() for n, t in p.items()}
    desc = C.swin_attn_join(C.swin_attn_norm(C.SWIN_NORM_LAYER, 1e-5, at["post_gamma"], at["post_beta"]),
                            C.swin_attn_norm(C.SWIN_NORM_RMS, 1e-5, at["pre_gamma"], at["pre_beta"]), at["scale"],
                            at["gate"], drop.desc, path.desc)
    dz = z.clone()
    # activations in place too: dx over dy, dz over z
    dx = dy.clone()
    C.swin_attn_join_bwd(rows, y, dz, desc, dx, dh, dx, dz, C.swin_attn_join_grads(*(at[n] for n in ALL)), ws)
    assert torch.equal(dx, want.dx) and torch.equal(dz, want.dz)
    for n in ALL:
        assert torch.equal(p[n], getattr(want, "d" + n)), n


def test_norm_gradients_over_their_parameters():
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm
    x, dh = (torch.randn(1, 900, 136, device="cuda") for _ in range(2))
    gamma, beta = (torch.randn(136, device="cuda") for _ in range(2))
    want = BlockNorm(136, dtype="f32").backward(x, dh, gamma, beta)
    rows = C.swin_attn_rows(1, 900, 136, C.SWIN_F32)
    ws = torch.empty(C.swin_attn_rows_workspace_bytes(rows), dtype=torch.uint8, device="cuda")
    norm = C.swin_attn_norm(C.SWIN_NORM_LAYER, 1e-5, gamma.data_ptr(), beta.data_ptr())
    dx = torch.empty_like(x)
    C.swin_attn_norm_bwd(rows, x, norm, dh, None, dx, gamma, beta, ws)
    assert torch.equal(dx, want[0]) and torch.equal(gamma, want[1]) and torch.equal(beta, want[2])


def test_a_refused_call_writes_nothing():
    """Without a gradient of h the pre norm's gradients are zeroed, but not by a call that is refused."""
    from shifted_window_attention_cyclic_gb300 import swin_attn as C
    x = torch.randn(2, 50, 64, device="cuda")
    grads = {n: torch.full((64,), 7.0, device="cuda") for n in ("pre_gamma", "pre_beta", "scale")}
    norm, none, off = C.swin_attn_norm(C.SWIN_NORM_LAYER, 1e-5, None, None), C.swin_attn_norm(0, 1e-5, None, None), C.swin_attn_drop(0.0, 0, None)
    rows, join = C.swin_attn_rows(2, 50, 64, C.SWIN_F32), C.swin_attn_join(none, norm, None, None, off, off)
    dx, dz = torch.empty_like(x), torch.empty_like(x)
    desc = C.swin_attn_join_grads(**{n: t.data_ptr() for n, t in grads.items()})
    with pytest.raises(C.SwinAttnError, match=r"\(%d\)" % C.SWIN_ERR_WORKSPACE):
        C.swin_attn_join_bwd(rows, x, x, join, x, None, dx, dz, desc, None)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in grads.values())
    ws = torch.empty(C.swin_attn_rows_workspace_bytes(rows), dtype=torch.uint8, device="cuda")
    C.swin_attn_join_bwd(rows, x, x, join, x, None, dx, dz, desc, ws)
    assert not grads["pre_gamma"].any() and not grads["pre_beta"].any() and grads["scale"].ne(7).all()
