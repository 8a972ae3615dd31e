"""The 64-bit reference of AdamW against what defines it: its first step, and the
table of e4m3."""
import pytest

torch = pytest.importorskip("torch")

from tests import optim_ref as ref  # noqa: E402


def test_e4m3_table():
    assert ref.E4M3.numel() == 127 and ref.E4M3[-1] == 448 and ref.E4M3[1] == 2.0**-9
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert torch.equal(codes.double(), ref.E4M3)
    x = torch.cat([torch.linspace(-448, 448, 501, dtype=torch.float64), ref.E4M3, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2])
    x = torch.cat([x, -x[501:]]).float()[:768].double()
    x[::256] = 448.0  # every unit's scale is one
    values, scale = ref.to_e4m3(x)
    assert (scale == 1).all() and torch.equal(values, x.to(torch.float8_e4m3fn).double())
    assert ref.to_e4m3(torch.tensor([448.0, 1e-9, 0.0], dtype=torch.float64), floor=True)[0].tolist() == [448.0, 2.0**-9, 0.0]


def test_adamw_first_step():
    """Of the first step m / (1 - b1) and v / (1 - b2) are g and g^2: the update is the sign of g."""
    w, g = torch.tensor([1.0, -2.0, 3.0], dtype=torch.float64), torch.tensor([0.5, -1e-3, 2.0], dtype=torch.float64)
    got, m, v = ref.adamw(w, g, torch.zeros(3).double(), torch.zeros(3).double(), 1, 0.1, 0.5, 0.9, 0.999, 1e-12)
    assert torch.allclose(got, w * 0.95 - 0.1 * torch.sign(g), rtol=1e-8)
    assert torch.allclose(m, 0.1 * g) and torch.allclose(v, 0.001 * g * g)
