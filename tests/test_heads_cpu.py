"""Refusals of the heads' entry points, on the CPU: every one returns or raises
before anything reaches a device."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import heads as H  # noqa: E402
from shifted_window_attention_cyclic_gb300 import swin_attn as C  # noqa: E402
from tests.test_rows_cpu import lib, norm  # noqa: E402,F401

A, B2, C3, D4, E5, F6 = (0x10000000 * (i + 1) for i in range(6))  # addresses that are never read
BAD, ALIGN, UNSUP = C.SWIN_ERR_INVALID_ARG, C.SWIN_ERR_ALIGNMENT, C.SWIN_ERR_UNSUPPORTED
FREQ, AXIS = np.ones(128, np.uint64), np.zeros(128, np.uint8)
BAD_AXIS = AXIS + np.uint8(2)


def rotary(dim=16, layout=0, amplitude=1.0, freq=FREQ, axis=AXIS, bits=0, shared=0, positions=None):
    return C.swin_attn_rotary(dim, layout, amplitude, None if freq is None else freq.ctypes.data,
                              None if axis is None else axis.ctypes.data, bits, shared, positions)


def heads(images=2, grid=(3, 5), head_dim=32, dtype=C.SWIN_BF16, rot=None, ndim=None):
    d = C.swin_attn_heads(images, len(grid) if ndim is None else ndim, (1, 1, 1), head_dim, dtype, rot or rotary())
    for a, g in enumerate(grid):
        d.grid[a] = g
    return d


def part(x=A, out=B2, n=2, rotate=1, nm=None, xs=64, os=64, dy=None, dys=64, dgamma=None, dbeta=None):
    return C.swin_attn_head_part(n, rotate, nm or norm(0), x, xs, dy, dys, out, os, dgamma, dbeta)


def parts(*p):
    return (C.swin_attn_head_part * len(p))(*p)


def fwd(lib, d, *p):
    return lib.swin_attn_heads_fwd(d, parts(*p), len(p), None)


def bwd(lib, d, *p, ws=0x70000000, n=1 << 22):
    return lib.swin_attn_heads_bwd(d, parts(*p), len(p), ws, n, None)


def test_bad_descriptors(lib):
    for d, code in ((heads(images=-1), BAD), (heads(ndim=0), BAD), (heads(ndim=4), BAD), (heads(grid=(3, -1)), BAD),
                    (heads(dtype=5), UNSUP), (heads(head_dim=0), UNSUP), (heads(head_dim=24), UNSUP),
                    (heads(head_dim=272), UNSUP), (heads(images=2**16, grid=(2**8, 2**8)), UNSUP),
                    (heads(images=2**40), UNSUP), (heads(grid=(2**30, 2**30, 2**30)), UNSUP),
                    (heads(rot=rotary(dim=-16)), BAD), (heads(rot=rotary(dim=24)), BAD), (heads(rot=rotary(dim=48)), BAD),
                    (heads(rot=rotary(layout=2)), BAD), (heads(rot=rotary(amplitude=float("nan"))), BAD),
                    (heads(rot=rotary(freq=None)), BAD), (heads(rot=rotary(axis=None)), BAD),
                    (heads(rot=rotary(axis=BAD_AXIS)), BAD), (heads(rot=rotary(bits=16)), BAD),
                    (heads(rot=rotary(shared=2)), BAD), (heads(rot=rotary(positions=E5)), BAD)):
        assert fwd(lib, d, part()) == code
        assert bwd(lib, d, part(x=None, dy=A)) == code
        assert lib.swin_attn_heads_workspace_bytes(d) == 0
    assert lib.swin_attn_heads_fwd(None, parts(part()), 1, None) == BAD
    assert lib.swin_attn_heads_fwd(heads(), None, 1, None) == BAD
    for count in (0, -1, 5):
        assert lib.swin_attn_heads_fwd(heads(), parts(*[part()] * 5), count, None) == BAD
    assert fwd(lib, heads(rot=rotary(bits=64)), part()) == BAD  # no positions
    assert fwd(lib, heads(rot=rotary(bits=64, positions=E5 + 4)), part()) == ALIGN
    assert fwd(lib, heads(rot=rotary(bits=32, positions=E5 + 2)), part()) == ALIGN


def test_bad_parts(lib):
    d = heads()
    for p, code in ((part(n=0), BAD), (part(n=65536), BAD), (part(n=513), UNSUP), (part(rotate=2), BAD), (part(x=None), BAD), (part(out=None), BAD),
                    (part(nm=norm(3)), BAD), (part(nm=norm(eps=0.0)), BAD), (part(nm=norm(eps=float("inf"))), BAD),
                    (part(nm=norm(0, gamma=C3)), BAD), (part(nm=norm(0, beta=C3)), BAD), (part(nm=norm(gamma=C3 + 2)), ALIGN),
                    (part(xs=63), BAD), (part(os=32), BAD), (part(xs=0), BAD), (part(xs=-64), BAD), (part(xs=2**61), BAD),
                    (part(xs=68), ALIGN), (part(os=66), ALIGN), (part(x=A + 8), ALIGN), (part(out=B2 + 2), ALIGN)):
        assert fwd(lib, d, p) == code, p
    n = norm(gamma=C3, beta=D4)
    for p, code in ((part(dy=None), BAD), (part(nm=n, dy=E5, x=None), BAD), (part(dy=E5, dgamma=F6), BAD),
                    (part(nm=n, dy=E5, dgamma=F6 + 2), ALIGN), (part(dy=E5, dys=60), BAD), (part(dy=E5, dys=68), ALIGN),
                    (part(dy=E5 + 4), ALIGN)):
        assert bwd(lib, d, p) == code, p
    assert bwd(lib, d, part(nm=n, dy=E5, dgamma=F6), ws=None) == C.SWIN_ERR_WORKSPACE


def test_overlaps(lib):
    """2 x 15 rows of 2 heads of 32: 128 bytes a row, 3840 in all."""
    d, g, b = heads(), C3, D4
    for p in (part(out=A + 16), part(out=A, os=72), part(out=A - 3824), part(nm=norm(gamma=B2)), part(nm=norm(beta=B2 + 3712))):
        assert fwd(lib, d, p) == BAD, p
    assert fwd(lib, heads(rot=rotary(bits=64, positions=B2 + 3832)), part()) == BAD
    # side by side in a packed tensor, and one row into its neighbour
    packed = lambda o, x=A, **k: part(x=x, out=o, xs=192, os=192, **k)  # noqa: E731
    assert fwd(lib, d, packed(B2), packed(B2 + 112, x=A + 128)) == BAD
    assert fwd(lib, d, packed(B2), packed(B2 + 128 + 384, x=A + 128), packed(B2 + 16, x=A + 256)) == BAD
    assert fwd(lib, d, packed(A), packed(C3, x=A)) == BAD  # another part's input
    assert fwd(lib, d, part(), part(x=C3)) == BAD  # one output twice
    n = norm(gamma=g, beta=b)
    back = lambda **k: bwd(lib, d, part(**{**dict(x=A, dy=E5, nm=n), **k}))  # noqa: E731
    for k in (dict(out=A + 16), dict(out=E5 + 128), dict(out=g), dict(dgamma=g + 4), dict(dgamma=b), dict(dbeta=g),
              dict(dgamma=F6, dbeta=F6 + 124), dict(dgamma=B2), dict(dgamma=A + 4), dict(dbeta=E5), dict(out=0x70000000)):
        assert back(**{"dgamma": F6 + 4096, **k}) == BAD, k
    two = bwd(lib, d, part(x=A, dy=E5, nm=n, dgamma=F6), part(x=C3 + 4096, out=D4 + 4096, dy=E5 + 4096, nm=n, dgamma=g))
    assert two == BAD  # over a gamma that another part reads


def test_nothing_to_do(lib):
    assert fwd(lib, heads(images=0), part(x=None, out=None)) == C.SWIN_OK
    assert fwd(lib, heads(grid=(0, 5)), part(x=None, out=None)) == C.SWIN_OK
    assert bwd(lib, heads(grid=(4, 0)), part(x=None, out=None)) == C.SWIN_OK


def test_bad_rotaries():
    for kw in (dict(dim=8), dict(dim=20), dict(dim=272), dict(dim=16, axes=0), dict(dim=16, axes=4),
               dict(dim=16, layout="quarter"), dict(dim=16, scaling="log"), dict(dim=16, factor=2.0),
               dict(dim=16, scaling="linear", factor=0.5), dict(dim=16, scaling="yarn", factor=2.0),
               dict(dim=16, base=0.0), dict(dim=16, frequencies=[1.0] * 7), dict(dim=16, axes=2, frequencies=[1.0] * 8),
               dict(dim=16, axes=2, frequencies=[1.0] * 8, axis_of=[2] * 8), dict(dim=16, frequencies=[float("nan")] * 8),
               dict(dim=16, axis_of=[0] * 8), dict(dim=16, frequencies=[1.0] * 8, scaling="linear", factor=2.0),
               dict(dim=16, amplitude=float("inf"))):
        with pytest.raises(ValueError):
            H.Rotary(**kw)
    for kw in (dict(heads=0, head_dim=32), dict(heads=2, head_dim=24), dict(heads=2, head_dim=272),
               dict(heads=2, head_dim=16, rotary=H.Rotary(32)), dict(heads=2, head_dim=32, rotary=16),
               dict(heads=2, head_dim=32, norm="batch"), dict(heads=2, head_dim=32, dtype="f16"),
               dict(heads=2, head_dim=32, eps=0.0), dict(heads=2, head_dim=32, kv_heads=0), dict(heads=65, head_dim=256)):
        with pytest.raises(ValueError):
            H.AttentionHeads(**kw)


def test_bad_calls():
    f = H.AttentionHeads(2, 32, H.Rotary(32, axes=2), norm="rms", dtype="f32")
    x = torch.zeros(1, 3, 5, 64)
    for call in (lambda: f.forward(x), lambda: f.forward(None), lambda: f.forward(x[0, 0, 0]),
                 lambda: f.forward(x[0]),  # one grid dimension, two axes
                 lambda: f.forward(x, positions=torch.zeros(15)), lambda: f.forward(x, positions=torch.zeros(3, 5, 1, dtype=torch.int64)),
                 lambda: f.backward(x), lambda: f.backward(x, packed=True), lambda: f.forward(x, k_gamma=torch.ones(32))):
        with pytest.raises(ValueError):
            call()


def test_rows_evenly_spaced():
    x = torch.zeros(2, 3, 5, 96)
    assert H._row_stride(x) == 96 and H._row_stride(x[..., 32:64]) == 96
    assert H._row_stride(x[:, :, :4, :32]) is None and H._row_stride(x[..., ::2]) is None
    assert H._row_stride(x[:, ::2, :, :]) is None and H._row_stride(x[:, :, ::5, :32]) == 480
    assert H._row_stride(x[:1, 1:2, 2:3, :32]) == 32 and H._row_stride(x.transpose(1, 2)) is None
    assert H._usable(x[..., 33:65]).is_contiguous() and H._usable(x[..., 32:64])._is_view()


class Heads:
    """u = x^2 for q and k, v copied; linear: u = 3 x."""

    def __init__(self, norm):
        self.norm = norm

    split = lambda self, qkv: qkv.split(4, -1)  # noqa: E731

    def forward(self, q, k, v, *params, positions=None):
        f = (lambda t: 3 * t) if self.norm == "none" else (lambda t: t * t)
        return f(q), f(k), v * 1

    def backward(self, dq, dk, dv, q, k, *params, positions=None, packed=False, want_params=True):
        g = (3 * dq, 3 * dk, dv) if self.norm == "none" else (2 * q * dq, 2 * k * dk, dv)
        return H.HeadGrads(*g, None, None, None, None, torch.cat(g, -1) if packed else None)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind", ["none", "rms"])
def test_autograd_function(kind, packed):
    leaf = torch.arange(1.0, 13.0).repeat(2, 1).requires_grad_(True)
    f = Heads(kind)

    def outputs():
        return H.attention_heads_packed(f, leaf) if packed else H.attention_heads(f, *f.split(leaf))

    slope = (torch.cat([2 * leaf[:, :8], torch.ones(2, 4)], -1) if kind == "rms" else
             torch.cat([torch.full((2, 8), 3.0), torch.ones(2, 4)], -1)).detach()
    assert torch.equal(torch.autograd.grad(torch.cat(outputs(), -1).sum(), leaf)[0], slope)
    g, = torch.autograd.grad(outputs()[0].sum(), leaf)  # outputs that nothing uses
    assert torch.equal(g[:, :4], slope[:, :4]) and (g[:, 4:] == 0).all()
    g, = torch.autograd.grad(torch.cat(outputs(), -1).square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
