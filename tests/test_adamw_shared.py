"""What DeviceAdamW refuses before any GPU work: tensors that share memory (all of them are updated at once), negative steps."""

import pytest

torch = pytest.importorskip("torch")
from int4_quantized_moe_amd import device  # noqa: E402


def test_tied_and_overlapping_tensors_are_refused():
    w = torch.zeros(600)
    for params in ({"a": w, "b": w}, {"a": w, "b": w.view(20, 30)}, {"a": w[:304], "b": w[300:]}, {"a": w, "b": w[8:12]}):
        with pytest.raises(ValueError, match="'a' and 'b' share memory|'b' and 'a' share memory"):
            device.DeviceAdamW(params)
    moment = torch.zeros(600)
    with pytest.raises(ValueError, match="share memory"):
        device.DeviceAdamW({"a": w}, state={"a": {"m": moment, "v": moment}})
    with pytest.raises(ValueError, match="share memory"):
        device.DeviceAdamW({"a": w}, state={"a": {"m": w}})
    both = w.bfloat16()
    with pytest.raises(ValueError, match="share memory"):
        device.DeviceAdamW({"a": both, "b": both}, states="e4m3", master=True)


def test_neighbours_and_empty_tensors_are_not():
    w = torch.zeros(600)
    o = device.DeviceAdamW({"a": w[:300], "b": w[300:], "c": w[:0], "d": w[300:300]}, states="e4m3")
    assert set(o.state) == {"a", "b", "c", "d"}


def test_a_negative_step_is_refused():
    """Its bias corrections would divide by 0."""
    with pytest.raises(ValueError, match="step must not be negative"):
        device.DeviceAdamW({"a": torch.zeros(8)}, step=-1)
