"""A dropout's settings, on the CPU."""
import pytest

pytest.importorskip("torch")

from shifted_window_attention_cyclic_gb300 import dropout as D  # noqa: E402


def test_settings_cannot_change_under_the_calls():
    """The library reads a descriptor made once: a rate set to 0 for an evaluation would still drop activations, and
    no longer attention probabilities."""
    state = D.DropoutState(3, device="cpu")
    drop = D.Dropout(state, 0.25, 7)
    for name, value in (("rate", 0.0), ("site", 8), ("state", D.DropoutState(4, device="cpu"))):
        with pytest.raises(AttributeError):
            setattr(drop, name, value)
    assert (drop.rate, drop.site, drop.state, drop.active) == (0.25, 7, state, True)
    assert (drop.desc.rate, drop.desc.site, drop.desc.state) == (0.25, 7, state.tensor.data_ptr())
    with pytest.raises(AttributeError):
        state.tensor = state.tensor.clone()
