"""What the autograd functions hand to the library and what they refuse, on the
CPU: the passes are stand-ins in torch operations, written as the kernels are
used (raw tensors in, tensors without a graph out)."""
import pytest

torch = pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import dropout as D  # noqa: E402
from shifted_window_attention_cyclic_gb300 import functional as F  # noqa: E402
from shifted_window_attention_cyclic_gb300 import residual as R  # noqa: E402


class Attention:
    """O = q k v and its gradient."""

    def forward(self, q, k, v, bias, land, dropout=None):
        return q * k * v, q.sum()

    def backward(self, q, k, v, dout, lse, bias, land, want_dbias=True, o=None, dropout=None):
        return dout * k * v, dout * q * v, dout * q * k, bias


class Norm:
    """h = x^2."""

    def forward(self, x, gamma, beta):
        return x * x

    def backward(self, x, dh, gamma, beta, want_params=True):
        return 2 * x * dh, gamma, beta


class Join:
    """y = x + z^2, as with a norm of z."""

    post, pre = "rms", "none"

    def forward(self, x, z, *params, drop=None, path=None):
        return x + z * z, None

    def backward(self, y, z, dy, dh, *params, drop=None, path=None, want_params=True):
        return R.JoinGrads(dy, 2 * z * dy, *params)


class PlainJoin:
    """y = x + 3 z: neither norms nor parameters."""

    post = pre = "none"

    def forward(self, x, z, *params, drop=None, path=None):
        return x + 3 * z, None

    def backward(self, y, z, dy, dh, *params, drop=None, path=None, want_params=True):
        return R.JoinGrads(dy, 3 * dy, *params)


def drop_every_second(x, drop, span=1):
    return x * torch.tensor([0.0, 2.0, 0.0, 2.0])


CALLS = {"attention": lambda x: F.swin_window_attention(Attention(), x, x, x),
         "norm": lambda x: R.block_norm(Norm(), x),
         "join": lambda x: R.residual_join(Join(), x, x)[0],
         "dropout": lambda x: D.dropout(x, None),
         "plain_join": lambda x: R.residual_join(PlainJoin(), x, x)[0]}


@pytest.mark.parametrize("name", ["attention", "norm", "join"])
def test_a_loss_over_the_gradient_is_refused(name):
    """f + |grad f|^2: the second term's gradient does not exist here, and leaving it out would be a wrong answer."""
    x = torch.full((4,), 2.0, requires_grad=True)
    y = CALLS[name](x)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (y.sum() + g.square().sum()).backward()


@pytest.mark.parametrize("name", sorted(CALLS))
def test_an_incoming_gradient_with_a_graph_is_refused(name, monkeypatch):
    monkeypatch.setattr(D, "apply_dropout", drop_every_second)
    x = torch.full((4,), 2.0, requires_grad=True)
    g, = torch.autograd.grad(CALLS[name](x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


@pytest.mark.parametrize("name,slope", [("dropout", [0.0, 2.0, 0.0, 2.0]), ("plain_join", [4.0] * 4)])
def test_a_linear_pass_has_a_constant_gradient(name, slope, monkeypatch):
    """There the second term adds nothing, and the answer is right."""
    monkeypatch.setattr(D, "apply_dropout", drop_every_second)
    x = torch.full((4,), 2.0, requires_grad=True)
    y = CALLS[name](x)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    assert g.tolist() == slope
    (y.sum() + g.square().sum()).backward()
    assert x.grad.tolist() == slope


@pytest.mark.parametrize("name,slope", [("attention", 12.0), ("norm", 4.0), ("join", 5.0)])
def test_first_derivatives_stay(name, slope):
    for graph in (False, True):
        x = torch.full((4,), 2.0, requires_grad=True)
        g, = torch.autograd.grad(CALLS[name](x).sum(), x, create_graph=graph)
        assert g.tolist() == [slope] * 4
