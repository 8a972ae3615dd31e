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


class Seen:
    """A stand-in's passes with the tensors that reach them."""

    def __init__(self, inner):
        self.inner, self.tensors = inner, []
        self.post, self.pre = getattr(inner, "post", None), getattr(inner, "pre", None)

    def _see(self, args):
        self.tensors += [a for a in args if isinstance(a, torch.Tensor) and a.dim()]

    def forward(self, *args, **kwargs):
        self._see(args)
        return self.inner.forward(*args, **kwargs)

    def backward(self, *args, **kwargs):
        self._see(args)
        return self.inner.backward(*args, **kwargs)


@pytest.mark.parametrize("name", ["attention", "norm", "join", "dropout"])
def test_tensors_off_a_16_byte_boundary_are_copied(name, monkeypatch):
    """A slice of a larger tensor, and a gradient that arrives as one (of a concatenation), may start anywhere; the
    library asks for 16 bytes, and the caller has no hand in where a gradient starts."""
    seen = Seen({"attention": Attention(), "norm": Norm(), "join": Join()}.get(name))

    def drop(x, drop, span=1):
        seen.tensors.append(x)
        return x * 2

    monkeypatch.setattr(D, "apply_dropout", drop)
    f = {"attention": lambda x: F.swin_window_attention(seen, x, x, x), "norm": lambda x: R.block_norm(seen, x),
         "join": lambda x: R.residual_join(seen, x, x)[0], "dropout": lambda x: D.dropout(x, None)}[name]
    grads = []
    for shift in (0, 1):  # elements of 4 bytes
        leaf = torch.cat([torch.zeros(shift), torch.arange(1.0, 5.0)]).requires_grad_(True)
        x = leaf[shift:]
        assert x.is_contiguous() and x.data_ptr() % 16 == 4 * shift
        y = torch.cat([torch.zeros(shift), f(x)])
        (y * torch.cat([torch.zeros(shift), torch.arange(5.0, 9.0)])).sum().backward()
        grads.append(leaf.grad[shift:])
    assert torch.equal(*grads)
    assert seen.tensors and all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in seen.tensors)
