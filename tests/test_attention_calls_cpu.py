"""What SwinWindowAttention hands to the library, on the CPU: the library's
calls are replaced by a record of their arguments."""
import types

import pytest

torch = pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import functional as F  # noqa: E402
from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState  # noqa: E402

CPU = torch.device("cpu")


@pytest.fixture
def attn(monkeypatch):
    """A module whose plan is never used, and the workspaces its backward calls got."""
    a = object.__new__(F.SwinWindowAttention)
    a.plan, a.device, a.torch_dtype, a.heads, a.has_land, a._ws = types.SimpleNamespace(), CPU, torch.float32, 2, False, None
    a.shape, a.lse_shape, a.bias_shape = (1, 4, 8, 64), (1, 2, 4, 8), (21, 2)
    a.got = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: CPU.index, raising=False)  # the current device
    monkeypatch.setattr(F.C, "swin_attn_workspace_bytes", lambda plan: 1000)
    monkeypatch.setattr(F.C, "swin_attn_bwd", lambda *args: a.got.append(args[12]))
    monkeypatch.setattr(F.C, "swin_attn_bwd_o", lambda *args: a.got.append(args[13]))
    monkeypatch.setattr(F.C, "swin_attn_bwd_dropout", lambda *args: a.got.append(args[13]))
    return a


@pytest.mark.parametrize("rate", [None, 0.0, 0.2])
@pytest.mark.parametrize("give_o", [False, True])
def test_backwards_that_may_overlap_share_no_workspace(attn, rate, give_o):
    """Two calls of one module, whose work another stream or a replayed graph may run at once."""
    x, lse = torch.zeros(attn.shape), torch.zeros(attn.lse_shape)
    drop = None if rate is None else Dropout(DropoutState(1, device=CPU), rate, 0)
    for _ in range(2):
        attn.backward(x, x, x, x, lse, o=x if give_o else None, dropout=drop)
    first, second = attn.got
    assert min(first.numel(), second.numel()) >= 1000
    assert first.data_ptr() != second.data_ptr()


@pytest.mark.parametrize("rate", [None, 0.2])
def test_what_a_call_allocates_belongs_to_its_stream(attn, rate, monkeypatch):
    """Memory is handed out again in the order of the stream it was allocated on: outputs and workspaces of a call on
    another stream than the current one have to come from that stream."""
    stream, now = types.SimpleNamespace(device=CPU), []

    class On:
        def __enter__(self):
            now.append(stream)

        def __exit__(self, *a):
            now.pop()

    monkeypatch.setattr(torch.cuda, "stream", lambda s: On())
    made = []
    for name in ("empty", "empty_like"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, real=real, **k: (made.append(list(now)), real(*a, **k))[1])
    calls = []
    for name in ("swin_attn_fwd", "swin_attn_fwd_dropout", "swin_attn_block_fwd"):
        monkeypatch.setattr(F.C, name, lambda *a: calls.append(list(now)))
    x, lse = torch.zeros(attn.shape), torch.zeros(attn.lse_shape)
    drop = None if rate is None else Dropout(DropoutState(1, device=CPU), rate, 0)
    attn.forward(x, x, x, stream=stream, dropout=drop)
    attn.backward(x, x, x, x, lse, stream=stream, dropout=drop)
    c = attn.shape[-1]
    vec, w = torch.zeros(c), torch.zeros(3 * c, c, dtype=torch.bfloat16)
    attn.block_forward(x, vec, vec, w, torch.zeros(3 * c), w[:c], vec, stream=stream)
    assert made and all(m == [stream] for m in made), made
    made.clear()
    attn.forward(x, x, x, dropout=drop)
    assert made and all(m == [] for m in made)
