"""The autograd functions around and of the window attention on the GPU: what
they refuse and what they take from a graph."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def calls():
    from shifted_window_attention_cyclic_gb300.dropout import Dropout, DropoutState, dropout
    from shifted_window_attention_cyclic_gb300.functional import SwinWindowAttention, swin_window_attention
    from shifted_window_attention_cyclic_gb300.residual import BlockNorm, ResidualJoin, block_norm, residual_join
    attn = SwinWindowAttention((9, 13), (4, 4), (2, 2), (0, 1), 2, 32, 1, "f32")
    drop = Dropout(DropoutState(5), 0.2, 1)
    return {"attention": lambda x: swin_window_attention(attn, x, x, x),
            "attention_dropout": lambda x: swin_window_attention(attn, x, x, x, dropout=drop),
            "norm": lambda x: block_norm(BlockNorm(64, dtype="f32"), x),
            "join": lambda x: residual_join(ResidualJoin(64, "rms", "layer", dtype="f32"), x, x, drop=drop)[1],
            "dropout": lambda x: dropout(x, drop)}


@pytest.mark.parametrize("name", ["attention", "attention_dropout", "norm", "join", "dropout"])
def test_second_derivatives_are_refused(name):
    x = torch.randn(1, 9, 13, 64, device="cuda", requires_grad=True)
    f = calls()[name]
    first, = torch.autograd.grad(f(x).sum(), x)
    for loss in (lambda y: y.sum(), lambda y: y.square().sum()):
        y = f(x)
        g, = torch.autograd.grad(loss(y), x, create_graph=True)
        if name == "dropout" and not g.requires_grad:  # linear: a constant, which adds nothing
            assert torch.equal(g, first)
            continue
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (y.sum() + g.square().sum()).backward()


@pytest.mark.parametrize("name", ["attention", "attention_dropout", "norm", "join", "dropout"])
def test_tensors_that_start_anywhere(name):
    """A slice as the input and a concatenation's slice as the gradient give what aligned tensors give."""
    f = calls()[name]
    x = torch.randn(1, 9, 13, 64, device="cuda")
    w = torch.randn(x.numel(), device="cuda")
    got = []
    for shift in (0, 1):
        leaf = torch.cat([x.new_zeros(shift), x.flatten()]).requires_grad_(True)
        y = torch.cat([x.new_zeros(shift), f(leaf[shift:].view(x.shape)).flatten()])
        (y[shift:] * w).sum().backward()
        got.append((y[shift:].detach(), leaf.grad[shift:]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
