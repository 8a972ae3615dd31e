"""Overlaps of outputs with what a call reads, on the CPU: an activation may be
written over an activation of the call and a parameter's gradient over that
parameter; everything else is refused before anything reaches a device."""
import pytest

pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import swin_attn as C  # noqa: E402
from tests.test_rows_cpu import A, B2, C3, D4, E5, F6, join, lib, norm, rows  # noqa: E402,F401


def test_outputs_over_parameters_and_states(lib):
    r, bad = rows(images=1, tokens=2, channels=32, dtype=C.SWIN_F32), C.SWIN_ERR_INVALID_ARG  # 256 bytes, parameters 128
    assert lib.swin_attn_norm_fwd(r, A, norm(gamma=B2 + 64), B2, None) == bad
    assert lib.swin_attn_norm_fwd(r, A, norm(beta=B2), B2, None) == bad
    assert lib.swin_attn_join_fwd(r, A, B2, join(scale=C3 + 128), C3, D4, None) == bad
    assert lib.swin_attn_join_fwd(r, A, B2, join(gate=D4 + 192), C3, D4, None) == bad
    drop = C.swin_attn_drop(0.1, 0, C3 + 16)
    assert lib.swin_attn_join_fwd(r, A, B2, join(drop=drop), C3, D4, None) == bad
    assert lib.swin_attn_join_fwd(r, A, B2, join(path=drop), C3, D4, None) == bad
    assert lib.swin_attn_dropout(C.SWIN_F32, 64, 1, A, drop, C3, None) == bad
    one = rows(images=1, tokens=1, channels=32, dtype=C.SWIN_F32)  # a row has a parameter's size
    assert lib.swin_attn_join_fwd(one, A, B2, join(scale=C3), C3, D4, None) == bad


def test_parameter_gradients_over_anything_but_their_parameter(lib):
    r, bad = rows(images=1, tokens=2, channels=32, dtype=C.SWIN_F32), C.SWIN_ERR_INVALID_ARG
    ws, P = 0x90000000, 0xA0000000
    nb = lambda n, dg, db, w=ws: lib.swin_attn_norm_bwd(r, A, n, B2, None, C3, dg, db, w, 1 << 20, None)  # noqa: E731
    assert nb(norm(), P, P) == bad  # both the same
    assert nb(norm(), P, P + 64) == bad
    assert nb(norm(), A + 16, None) == bad  # over x
    assert nb(norm(), None, C3 + 252) == bad  # over dx
    assert nb(norm(gamma=P), P + 4, None) == bad  # partly over its parameter
    assert nb(norm(gamma=P), None, P) == bad  # over another parameter
    assert nb(norm(), ws + 256, None) == bad  # over the workspace
    assert nb(norm(), P, None, A & ~255) == bad  # the workspace over x
    j = join(post=norm(gamma=P, beta=P + 0x1000), pre=norm(gamma=P + 0x2000, beta=P + 0x3000), scale=P + 0x4000,
             gate=P + 0x5000)
    names = ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "scale", "gate")

    def jb(**g):
        return lib.swin_attn_join_bwd(r, A, B2, j, C3, D4, E5, F6, C.swin_attn_join_grads(**g), ws, 1 << 20, None)

    for k, name in enumerate(names):
        for at in [P + 0x1000 * o for o in range(6) if o != k] + [P + 0x1000 * k + 4, A, B2, C3 + 128, D4, E5, F6, ws]:
            assert jb(**{name: at}) == bad, (name, hex(at))
        other = names[(k + 1) % 6]
        assert jb(**{name: P + 0x8000, other: P + 0x8000 + 124}) == bad
    drop = C.swin_attn_drop(0.1, 0, P + 0x9000)
    j = join(drop=drop, scale=P)
    assert jb(scale=P + 0x9000) == bad


def test_nothing_overlaps_an_empty_tensor(lib):
    """Without rows the activations are empty, wherever their pointers point. (Refused later, for want of a workspace.)"""
    r, P = rows(images=2, tokens=0, channels=32, dtype=C.SWIN_F32), 0xA0000000
    assert lib.swin_attn_norm_bwd(r, P + 16, norm(), P + 32, None, P + 64, P, None, None, 0, None) != C.SWIN_ERR_INVALID_ARG
    g = C.swin_attn_join_grads(scale=P)
    assert lib.swin_attn_join_bwd(r, P + 16, B2, join(), C3, D4, P + 32, P + 64, g, None, 0, None) != C.SWIN_ERR_INVALID_ARG
