"""Backwards of one attention module that run at the same time: on two streams
and as two captured graphs, against the same calls alone."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

GEOMETRY = [(32, (48, 96), (4, 8), "bf16"), (128, (64, 96), (16, 16), "bf16"), (16, (32, 64), (4, 8), "f32")]


def setup(head_dim, grid, window, dtype, rate):
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
    attn = SwinWindowAttention(grid, window, (2, 4), (0, 1), 2, head_dim, 1, dtype)
    gen = torch.Generator().manual_seed(3)
    q, k, v, *douts = (torch.randn(attn.shape, generator=gen).to(attn.torch_dtype).cuda() for _ in range(5))
    bias = (torch.randn(attn.bias_shape, generator=gen) * 0.1).cuda()
    drop = Dropout(DropoutState(9, 2), rate, 4) if rate is not None else None
    o, lse = attn.forward(q, k, v, bias, dropout=drop)

    def backward(dout, stream=None):
        return attn.backward(q, k, v, dout, lse, bias, o=o, dropout=drop, stream=stream)

    return douts, backward


def same(got, want, head_dim):
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    if head_dim == 128:  # its dBias is summed by atomics: fp32 sums of some thousand terms in another order
        assert (got[3] - want[3]).norm() <= 1e-4 * want[3].norm()
    else:
        assert torch.equal(got[3], want[3])


@pytest.mark.parametrize("rate", [None, 0.0, 0.2])
@pytest.mark.parametrize("head_dim,grid,window,dtype", GEOMETRY, ids=lambda x: str(x))
def test_two_streams_and_two_graphs(head_dim, grid, window, dtype, rate):
    douts, backward = setup(head_dim, grid, window, dtype, rate)
    want = [[t.clone() for t in backward(d)] for d in douts]
    assert not torch.equal(want[0][3], want[1][3])
    side = [torch.cuda.Stream() for _ in douts]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, s in enumerate(side):
            got[k].append(backward(douts[k], s))
    torch.cuda.synchronize()
    for k in range(2):
        for g in got[k]:
            same(g, want[k], head_dim)

    graphs = []
    for d in douts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = backward(d)
        graphs.append((g, out))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (g, _) in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for k, (_, out) in enumerate(graphs):
            same(out, want[k], head_dim)


def stream_of(t):
    """The stream that the memory of `t` was allocated on."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("rate", [None, 0.2])
def test_outputs_belong_to_the_stream_they_are_written_on(rate):
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
    attn = SwinWindowAttention((16, 32), (4, 8), (2, 4), (0, 1), 2, 32)
    q, k, v, dout = (torch.randn(attn.shape, device="cuda").bfloat16() for _ in range(4))
    bias = attn.new_bias()
    drop = Dropout(DropoutState(9), rate, 4) if rate is not None else None
    o, lse = attn.forward(q, k, v, bias, dropout=drop)
    want = (o, lse) + attn.backward(q, k, v, dout, lse, bias, dropout=drop)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = attn.forward(q, k, v, bias, dropout=drop, stream=side)
    got = (o2, lse2) + attn.backward(q, k, v, dout, lse2, bias, dropout=drop, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert {stream_of(t) for t in got} == {side.cuda_stream}
    assert side.cuda_stream not in {stream_of(t) for t in want}
