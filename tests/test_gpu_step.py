"""A whole training step of an attention block, as its parts are used together: the
packed projection, head norm with rotary positions, the window attention with
dropped probabilities, the residual join, the backward of all of them and the
parameters' update; eager, and captured and replayed."""
import gc

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def no_memory_kept():
    """Give the allocator's blocks back: a later test counts what its calls hold, and a cached block may be the larger one."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


GRID, HEADS, HD = (12, 20), 2, 32
C = HEADS * HD


class Block:
    def __init__(self, bits, seed=3):
        from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState
        from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention
        from shifted_window_attention_cyclic_gb300.heads import AttentionHeads, Rotary
        from shifted_window_attention_cyclic_gb300.optim import AdamW
        from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin
        gen = torch.Generator().manual_seed(seed)
        self.state = DropoutState(5)
        self.drop = [Dropout(self.state, 0.1, site) for site in (0, 1)]
        self.attn = SwinWindowAttention(GRID, (4, 8), (2, 4), (0, 1), HEADS, HD, 2, "bf16")
        self.heads = AttentionHeads(HEADS, HD, Rotary(HD, axes=2), norm="rms")
        self.norm, self.join = BlockNorm(C), ResidualJoin(C, pre="layer")

        def leaf(*shape, std=1.0, mean=0.0, dtype=torch.float32):
            return (torch.randn(shape, generator=gen) * std + mean).to(dtype).cuda().requires_grad_(True)

        self.w_qkv, self.w_o = leaf(3 * C, C, std=0.1, dtype=torch.bfloat16), leaf(C, C, std=0.1, dtype=torch.bfloat16)
        self.vecs = [leaf(C, std=0.1, mean=1.0), leaf(C, std=0.1), leaf(HD, std=0.1, mean=1.0), leaf(HD, std=0.1, mean=1.0),
                     leaf(*self.attn.bias_shape, std=0.02), leaf(C, std=0.1, mean=0.3), leaf(C, std=0.1, mean=1.0), leaf(C, std=0.1)]
        self.x = torch.randn(2, *GRID, C, generator=gen).bfloat16().cuda()
        self.dy = torch.randn(2, *GRID, C, generator=gen).bfloat16().cuda()
        self.opt = AdamW([{"params": [self.w_qkv, self.w_o], "weight_decay": 0.1},
                          {"params": self.vecs, "weight_decay": 0.0}], lr=1e-2, state_bits=bits, max_norm=1.0)

    def forward(self):
        from shifted_window_attention_cyclic_gb300.functional import swin_window_attention
        from shifted_window_attention_cyclic_gb300.heads import attention_heads_packed
        from shifted_window_attention_cyclic_gb300.residual import block_norm, residual_join
        g1, b1, gq, gk, bias, scale, g2, b2 = self.vecs
        h = block_norm(self.norm, self.x, g1, b1)
        q, k, v = attention_heads_packed(self.heads, h @ self.w_qkv.t(), q_gamma=gq, k_gamma=gk)
        o = swin_window_attention(self.attn, q, k, v, bias, dropout=self.drop[0])
        return residual_join(self.join, self.x, o @ self.w_o.t(), scale=scale, pre_gamma=g2, pre_beta=b2, drop=self.drop[1])

    def step(self):
        y, h = self.forward()
        grads = torch.autograd.grad([y, h], self.opt.params, [self.dy, self.dy])
        self.opt.step(grads)
        self.state.advance()
        return y

    def everything(self):
        return [p.detach().clone() for p in self.opt.params] + [t.clone().reshape(-1).view(torch.uint8) for t in (
            self.opt.m, self.opt.v, self.opt.master, self.opt.steps, self.opt.grad_norm)]


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_are_the_eager_ones(bits):
    eager, captured = Block(bits), Block(bits)
    for _ in range(2):
        eager.step()
    side = torch.cuda.Stream()  # the first steps of the captured block run on the stream that captures
    with torch.cuda.stream(side):
        for _ in range(2):
            captured.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager.everything(), captured.everything()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured.step()
    for k in range(3):
        for b in (eager, captured):
            b.opt.lr.fill_(1e-2 / (k + 1))
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager.everything(), captured.everything())), k
    assert int(captured.opt.steps) == 5


def test_gradients_against_plain_operations():
    """The chain's gradients against torch's own of the same formulas in fp32, without dropout; each operator is held to its
    reference elsewhere, here what is handed from one to the next."""
    from tests import heads_ref as ref
    b = Block(32)
    b.drop = [None, None]
    y, h = b.forward()
    got = torch.autograd.grad([y, h], b.opt.params, [b.dy, b.dy])

    from shifted_window_attention_cyclic_gb300 import swin_attn as A
    win_src, region, _, relidx = A.swin_attn_plan_tables(b.attn.plan)
    src, reg, rel = (torch.from_numpy(t).long().cuda() for t in (win_src, region, relidx))
    w_qkv, w_o = (w.detach().float().requires_grad_(True) for w in (b.w_qkv, b.w_o))
    vecs = [v.detach().clone().requires_grad_(True) for v in b.vecs]
    g1, b1, gq, gk, bias, scale, g2, b2 = vecs
    x, n = b.x.float(), GRID[0] * GRID[1]
    norm = torch.nn.functional.layer_norm
    hh = norm(x, (C,), g1, b1, 1e-5)
    q, k, v = (hh @ w_qkv.t()).view(2, n, 3, HEADS, HD).unbind(2)
    t = ref.turns(ref.grid_positions(1, GRID), b.heads.rotary.frequencies, b.heads.rotary.axis_of).float().cuda()

    def turned(u, gamma):
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-5) * gamma
        a, c = u[..., :HD // 2], u[..., HD // 2:]
        return torch.cat([a * t.cos() - c * t.sin(), a * t.sin() + c * t.cos()], -1)

    q, k, v = (u[:, src.clamp(min=0)].transpose(2, 3) for u in (turned(q, gq), turned(k, gk), v))  # [2, nwin, H, n, hd]
    live = (src >= 0)[:, None, :] & (src >= 0)[:, :, None] & (reg[:, None, :] == reg[:, :, None])
    s = q @ k.transpose(-1, -2) * HD**-0.5 + bias[rel].permute(2, 0, 1)
    p = s.masked_fill(~live[None, :, None], -1e30).softmax(-1)
    o = (p @ v).transpose(2, 3).reshape(2, src.shape[0], src.shape[1], C)
    tokens = torch.zeros(2, n, C, device="cuda").index_copy(1, src[src >= 0], o[:, src >= 0])
    y32 = x + scale * (tokens.view(x.shape) @ w_o.t())
    want = torch.autograd.grad([y32, norm(y32, (C,), g2, b2, 1e-5)], [w_qkv, w_o] + vecs, [b.dy.float()] * 2)
    # some eight tensors of the chain are rounded to bf16, each by up to 2^-8 a value, and their errors add as vectors at most
    for i, (a, w) in enumerate(zip(got, want)):
        assert (a.float() - w).norm() <= 8 * 2.0**-8 * w.norm(), i
