"""Calls whose outputs exist already, from a host thread that has made no CUDA
call yet (an autograd worker, a data-parallel replica's thread): the library
binds the device's context itself."""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def in_new_thread(f):
    got = []

    def body():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001 (the assertion below shows it)
            got.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    assert not isinstance(got[0], Exception), got[0]
    return got[0]


@pytest.mark.parametrize("head_dim,window,dtype", [(32, (4, 8), "bf16"), (128, (16, 16), "bf16"), (16, (4, 8), "f32")])
@pytest.mark.parametrize("rate", [0.0, 0.2])
def test_attention_from_a_fresh_thread(head_dim, window, dtype, rate):
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
    attn = SwinWindowAttention((20, 36), window, (2, 4), (0, 1), 2, head_dim, 1, dtype)
    q, k, v, do = (torch.randn(attn.shape, device="cuda").to(attn.torch_dtype) for _ in range(4))
    drop = Dropout(DropoutState(3), rate, 1)
    o, lse = attn.forward(q, k, v, dropout=drop)
    want = attn.backward(q, k, v, do, lse, dropout=drop, want_dbias=False)
    outs = [torch.empty_like(q) for _ in range(4)]
    lse2 = torch.empty_like(lse)
    attn.workspace()
    torch.cuda.synchronize()
    in_new_thread(lambda: attn.forward(q, k, v, o=outs[0], lse=lse2, dropout=drop))
    in_new_thread(lambda: attn.backward(q, k, v, do, lse, dq=outs[1], dk=outs[2], dv=outs[3], dropout=drop, want_dbias=False))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], o) and torch.equal(lse2, lse)
    assert all(torch.equal(a, b) for a, b in zip(outs[1:], want))


def test_rows_from_a_fresh_thread():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, apply_dropout
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm
    x, h = torch.randn(2, 50, 96, device="cuda"), torch.empty(2, 50, 96, device="cuda")
    drop = Dropout(DropoutState(3), 0.2, 1)
    norm, want = BlockNorm(96, dtype="f32"), apply_dropout(x, drop)
    torch.cuda.synchronize()
    in_new_thread(lambda: norm.forward(x, h=h))
    assert torch.equal(h, norm.forward(x))
    in_new_thread(lambda: apply_dropout(x, drop, out=h))
    assert torch.equal(h, want)
