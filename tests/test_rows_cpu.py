"""Refusals of the norm, join and dropout entry points, on the CPU: every one
returns or raises before anything reaches a device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import dropout as D  # noqa: E402
from shifted_window_attention_cyclic_gb300 import residual as R  # noqa: E402
from shifted_window_attention_cyclic_gb300 import swin_attn as C  # noqa: E402

A, B2, C3, D4, E5, F6 = (0x10000000 * (i + 1) for i in range(6))  # addresses that are never read


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return C.load_library()


def rows(images=2, tokens=5, channels=32, dtype=C.SWIN_BF16):
    return C.swin_attn_rows(images, tokens, channels, dtype)


def norm(kind=C.SWIN_NORM_LAYER, eps=1e-5, gamma=None, beta=None):
    return C.swin_attn_norm(kind, eps, gamma, beta)


def join(post=None, pre=None, scale=None, gate=None, drop=None, path=None):
    none = C.swin_attn_drop(0.0, 0, None)
    return C.swin_attn_join(post or norm(0), pre or norm(), scale, gate, drop or none, path or none)


def test_bad_rows(lib):
    n = norm()
    for bad, code in ((rows(images=-1), C.SWIN_ERR_INVALID_ARG), (rows(tokens=-1), C.SWIN_ERR_INVALID_ARG),
                      (rows(dtype=9), C.SWIN_ERR_UNSUPPORTED), (rows(channels=0), C.SWIN_ERR_UNSUPPORTED),
                      (rows(channels=12), C.SWIN_ERR_UNSUPPORTED), (rows(channels=8200), C.SWIN_ERR_UNSUPPORTED),
                      (rows(images=2**20, tokens=2**20), C.SWIN_ERR_UNSUPPORTED),
                      (rows(tokens=2**40), C.SWIN_ERR_UNSUPPORTED)):
        assert lib.swin_attn_norm_fwd(bad, A, n, B2, None) == code
        assert lib.swin_attn_norm_bwd(bad, A, n, B2, None, C3, None, None, None, 0, None) == code
        assert lib.swin_attn_join_fwd(bad, A, B2, join(), C3, D4, None) == code
        assert lib.swin_attn_join_bwd(bad, A, B2, join(), C3, D4, E5, F6, C.swin_attn_join_grads(), None, 0,
                                      None) == code
        assert lib.swin_attn_rows_workspace_bytes(bad) == 0
    assert lib.swin_attn_norm_fwd(None, A, n, B2, None) == C.SWIN_ERR_INVALID_ARG


def test_bad_norm_arguments(lib):
    r, f = rows(), lib.swin_attn_norm_fwd
    assert f(r, A, None, B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, norm(0), B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, norm(3), B2, None) == C.SWIN_ERR_INVALID_ARG
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert f(r, A, norm(eps=eps), B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, None, norm(), B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, norm(), None, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, norm(), A + 16, None) == C.SWIN_ERR_INVALID_ARG  # partial overlap
    assert f(r, A + 8, norm(), B2, None) == C.SWIN_ERR_ALIGNMENT
    assert f(r, A, norm(), B2 + 2, None) == C.SWIN_ERR_ALIGNMENT
    assert f(r, A, norm(gamma=C3 + 2), B2, None) == C.SWIN_ERR_ALIGNMENT
    b = lib.swin_attn_norm_bwd
    assert b(r, A, norm(), None, None, C3, None, None, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, norm(), B2, None, None, None, None, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, norm(), B2, C3 + 16, C3, None, None, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, norm(), B2, None, C3, D4 + 1, None, None, 0, None) == C.SWIN_ERR_ALIGNMENT


def test_bad_join_arguments(lib):
    r, f = rows(), lib.swin_attn_join_fwd
    assert f(r, A, B2, None, C3, D4, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, B2, join(), C3, None, None) == C.SWIN_ERR_INVALID_ARG  # the pre norm has no output
    assert f(r, A, B2, join(pre=norm(0)), C3, D4, None) == C.SWIN_ERR_INVALID_ARG  # an output has no norm
    assert f(r, A, None, join(), C3, D4, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, B2, join(), C3, C3, None) == C.SWIN_ERR_INVALID_ARG  # outputs overlap
    assert f(r, A, B2, join(), A + 32, D4, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, B2, join(), C3, B2 + 32, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, B2 + 4, join(), C3, D4, None) == C.SWIN_ERR_ALIGNMENT
    assert f(r, A, B2, join(gate=E5 + 2), C3, D4, None) == C.SWIN_ERR_ALIGNMENT
    for rate in (-0.1, 1.0, 1.5, float("nan"), 1 - 2**-18):
        d = C.swin_attn_drop(rate, 0, F6)
        assert f(r, A, B2, join(drop=d), C3, D4, None) == C.SWIN_ERR_INVALID_ARG
        assert f(r, A, B2, join(path=d), C3, D4, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, B2, join(drop=C.swin_attn_drop(0.1, 0, None)), C3, D4, None) == C.SWIN_ERR_INVALID_ARG
    assert f(r, A, B2, join(drop=C.swin_attn_drop(0.1, 0, F6 + 4)), C3, D4, None) == C.SWIN_ERR_ALIGNMENT
    b, none = lib.swin_attn_join_bwd, C.swin_attn_join_grads()
    assert b(r, A, B2, join(), None, None, E5, F6, none, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, B2, join(), C3, D4, E5, F6, None, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, None, B2, join(), C3, D4, E5, F6, none, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, None, join(post=norm()), C3, D4, E5, F6, none, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, B2, join(), C3, D4, E5, E5, none, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, B2, join(pre=norm(0)), C3, D4, E5, F6, none, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    for g in (C.swin_attn_join_grads(post_gamma=64), C.swin_attn_join_grads(gate=64)):
        assert b(r, A, B2, join(), C3, D4, E5, F6, g, None, 0, None) == C.SWIN_ERR_INVALID_ARG
    assert b(r, A, B2, join(pre=norm(0)), C3, None, E5, F6, C.swin_attn_join_grads(pre_gamma=64), None, 0,
             None) == C.SWIN_ERR_INVALID_ARG


def test_bad_dropout_arguments(lib):
    f, d = lib.swin_attn_dropout, C.swin_attn_drop(0.1, 0, F6)
    assert f(C.SWIN_BF16, -1, 1, A, d, B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(C.SWIN_BF16, 64, 0, A, d, B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(5, 64, 1, A, d, B2, None) == C.SWIN_ERR_UNSUPPORTED
    assert f(C.SWIN_F32, 64, 1, None, d, B2, None) == C.SWIN_ERR_INVALID_ARG
    assert f(C.SWIN_F32, 64, 1, A, d, A + 64, None) == C.SWIN_ERR_INVALID_ARG
    assert f(C.SWIN_F32, 64, 1, A + 4, d, B2, None) == C.SWIN_ERR_ALIGNMENT
    assert f(C.SWIN_F32, 64, 1, A, C.swin_attn_drop(1.0, 0, F6), B2, None) == C.SWIN_ERR_INVALID_ARG
    # nothing to do: nothing is read, nothing launched
    assert f(C.SWIN_F32, 0, 1, None, d, None, None) == C.SWIN_OK
    assert lib.swin_attn_norm_fwd(rows(tokens=0), None, norm(), None, None) == C.SWIN_OK
    assert lib.swin_attn_join_fwd(rows(images=0), None, None, join(), None, None, None) == C.SWIN_OK


def test_attention_dropout_refusals(lib):
    d = C.swin_attn_drop(0.1, 0, F6)
    assert lib.swin_attn_fwd_dropout(None, *([None] * 7), d, None) == C.SWIN_ERR_INVALID_ARG
    assert lib.swin_attn_bwd_dropout(None, *([None] * 13), 0, d, None) == C.SWIN_ERR_INVALID_ARG


def test_python_refusals():
    state = D.DropoutState(2**64 - 1, device="cpu")
    assert state.tensor.tolist() == [-1, 0]
    state.advance()
    assert state.tensor.tolist() == [-1, 1]
    for seed in (-1, 2**64):
        with pytest.raises(ValueError, match="seed"):
            D.DropoutState(seed, device="cpu")
    for rate in (-0.1, 1.0, 1 - 2**-18, float("nan")):
        with pytest.raises(ValueError, match="rate"):
            D.Dropout(state, rate, 0)
    for site in (-1, 2**32, 0.5):
        with pytest.raises(ValueError, match="site"):
            D.Dropout(state, 0.1, site)
    with pytest.raises(ValueError, match="state"):
        D.Dropout(state.tensor, 0.1, 0)
    assert not D.Dropout(state, 2**-18, 0).active and D.Dropout(state, 2**-16, 0).active
    x = torch.zeros(2, 3, 32)
    with pytest.raises(ValueError, match="CUDA"):
        D.apply_dropout(x, None)
    with pytest.raises(ValueError, match="x: expected"):
        D.apply_dropout(x.half(), None)
    for bad in (0, 12, 8200):
        with pytest.raises(ValueError, match="channels"):
            R.BlockNorm(bad)
    with pytest.raises(ValueError, match="kind"):
        R.BlockNorm(32, "none")
    with pytest.raises(ValueError, match="eps"):
        R.BlockNorm(32, eps=0.0)
    with pytest.raises(ValueError, match="dtype"):
        R.ResidualJoin(32, dtype="fp16")
    with pytest.raises(ValueError, match="post"):
        R.ResidualJoin(32, post="batch")
    with pytest.raises(ValueError, match="CUDA"):
        R.BlockNorm(32, dtype="f32").forward(x)
