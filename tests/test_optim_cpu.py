"""Refusals of the optimiser's entry points, on the CPU: every one returns or
raises before anything reaches a device."""
import pytest

torch = pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import optim as O  # noqa: E402
from shifted_window_attention_cyclic_gb300 import swin_attn as C  # noqa: E402
from tests.test_rows_cpu import lib  # noqa: E402,F401

BAD, ALIGN, UNSUP, SPACE = C.SWIN_ERR_INVALID_ARG, C.SWIN_ERR_ALIGNMENT, C.SWIN_ERR_UNSUPPORTED, C.SWIN_ERR_WORKSPACE
P, M, G, S, V, MS, VS, LR, T, N, WS = (0x10000000 * (i + 1) for i in range(11))  # addresses that are never read


def param(n=1000, dtype=C.SWIN_F32, grad_dtype=C.SWIN_F32, p=P, master=None, grad=G, m=S, v=V, ms=None, vs=None, decay=0.1):
    return C.swin_attn_param(n, dtype, grad_dtype, p, master, grad, m, v, ms, vs, decay)


def adamw(b1=0.9, b2=0.999, eps=1e-8, max_norm=0.0, bits=32, lr=LR, steps=T, norm=None):
    return C.swin_attn_adamw(b1, b2, eps, max_norm, bits, lr, steps, norm)


def step(lib, o, *p, ws=WS, n=1 << 20, count=None):
    a = (C.swin_attn_param * max(len(p), 1))(*p)
    return lib.swin_attn_adamw_step(o, a, len(p) if count is None else count, ws, n, None)


def norm(lib, *p, out=N, ws=WS, n=1 << 20):
    return lib.swin_attn_grad_norm((C.swin_attn_param * max(len(p), 1))(*p), len(p), out, ws, n, None)


def test_the_table_is_the_library_s():
    import ctypes
    assert O._PARAM.itemsize == ctypes.sizeof(C.swin_attn_param)
    for name, _ in C.swin_attn_param._fields_:
        assert O._PARAM.fields[name][1] == getattr(C.swin_attn_param, name).offset, name


def test_bad_optimisers(lib):
    nan, inf = float("nan"), float("inf")
    for o, code in ((None, BAD), (adamw(b1=-0.1), BAD), (adamw(b1=1.0), BAD), (adamw(b2=1.0), BAD), (adamw(b2=nan), BAD),
                    (adamw(eps=0.0), BAD), (adamw(eps=-1.0), BAD), (adamw(eps=inf), BAD), (adamw(eps=1e-60), BAD),
                    (adamw(eps=1e60), BAD), (adamw(max_norm=-1.0), BAD), (adamw(max_norm=inf), BAD),
                    (adamw(max_norm=nan), BAD), (adamw(norm=N), BAD), (adamw(bits=16), UNSUP), (adamw(lr=None), BAD),
                    (adamw(steps=None), BAD), (adamw(lr=LR + 2), ALIGN), (adamw(steps=T + 4), ALIGN),
                    (adamw(max_norm=1.0, norm=N + 1), ALIGN)):
        assert step(lib, o, param()) == code
    assert step(lib, adamw(), param(), ws=None) == SPACE
    assert step(lib, adamw(), param(), n=lib.swin_attn_adamw_workspace_bytes() - 1) == SPACE
    assert step(lib, adamw(), param(), ws=WS + 16) == ALIGN
    assert step(lib, adamw(), param(), count=-1) == BAD
    assert lib.swin_attn_adamw_step(adamw(), None, 1, WS, 1 << 20, None) == BAD


def test_bad_tensors(lib):
    for p, code in ((param(n=-1), BAD), (param(dtype=7), UNSUP), (param(grad_dtype=7), UNSUP), (param(decay=-1.0), BAD),
                    (param(decay=float("nan")), BAD), (param(p=None), BAD), (param(m=None), BAD), (param(v=None), BAD),
                    (param(master=M), BAD), (param(dtype=C.SWIN_BF16), BAD), (param(ms=MS), BAD), (param(vs=VS), BAD),
                    (param(p=P + 2), ALIGN), (param(grad=G + 2), ALIGN), (param(m=S + 2), ALIGN), (param(v=V + 1), ALIGN),
                    (param(dtype=C.SWIN_BF16, master=M + 2), ALIGN), (param(dtype=C.SWIN_BF16, p=P + 1, master=M), ALIGN),
                    (param(grad_dtype=C.SWIN_BF16, grad=G + 1), ALIGN), (param(n=2**39), UNSUP)):
        assert step(lib, adamw(), p) == code, p
    assert step(lib, adamw(), param(n=2**38), param(n=2**38)) == UNSUP
    for p, code in ((param(), BAD), (param(ms=MS), BAD), (param(vs=VS), BAD), (param(ms=MS + 2, vs=VS), ALIGN),
                    (param(ms=MS, vs=VS + 1), ALIGN)):
        assert step(lib, adamw(bits=8), p) == code, p


def test_overlaps(lib):
    o = adamw(max_norm=1.0, norm=N)
    for p in (param(m=P), param(m=P + 3996), param(v=S + 8), param(grad=P), param(grad=P - 3996), param(grad=S + 3996),
              param(p=LR - 8), param(m=T - 3996), param(v=N), param(v=WS + 64), param(grad=WS + 128), param(grad=T),
              param(dtype=C.SWIN_BF16, master=P + 1996)):
        assert step(lib, o, p) == BAD, p
    far = 0x2000
    other = dict(p=P + far, grad=G + far, m=S + far, v=V + far)
    for k, at in (("p", P), ("p", P + 3996), ("m", S), ("v", V + 4), ("m", P + 400), ("grad", P + 4), ("grad", V)):
        assert step(lib, o, param(), param(**{**other, k: at})) == BAD, k
    eight = adamw(bits=8)
    for p in (param(ms=MS, vs=MS + 12), param(ms=S, vs=VS), param(ms=MS, vs=V + 996), param(m=S, v=S + 999, ms=MS, vs=VS)):
        assert step(lib, eight, p) == BAD, p


def test_bad_norms(lib):
    for p, code in ((param(n=-1), BAD), (param(grad_dtype=3), UNSUP), (param(grad=G + 1), ALIGN), (param(n=2**40), UNSUP)):
        assert norm(lib, p) == code
    assert norm(lib, param(), out=None) == BAD and norm(lib, param(), out=N + 2) == ALIGN
    assert norm(lib, param(), ws=None) == SPACE and norm(lib, param(), n=64) == SPACE and norm(lib, param(), ws=WS + 8) == ALIGN
    assert norm(lib, param(), out=G + 16) == BAD and norm(lib, param(grad=WS)) == BAD and norm(lib, param(), out=WS + 512) == BAD


def test_bad_calls():
    x = torch.zeros(4)
    for call in (lambda: O.grad_norm([]), lambda: O.grad_norm([x]), lambda: O.grad_norm([None]), lambda: O.AdamW([]),
                 lambda: O.AdamW([x]), lambda: O.AdamW([None]), lambda: O.AdamW(x), lambda: O.AdamW([x], lr=float("nan")),
                 lambda: O.AdamW([x], betas=(0.9, 1.0)), lambda: O.AdamW([x], betas=(0.9,)), lambda: O.AdamW([x], eps=0.0),
                 lambda: O.AdamW([x], weight_decay=-0.1), lambda: O.AdamW([{"params": [x], "weight_decay": float("inf")}]),
                 lambda: O.AdamW([x], state_bits=16), lambda: O.AdamW([x], max_norm=0.0), lambda: O.AdamW([x.double()])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="rows"):
        O.AdamW(x)
