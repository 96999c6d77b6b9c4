"""CPU: what the classes of the norms, of AdamW and of the experts for a few tokens do around the library's calls: the
tensors' GPU made current, the streams and workspaces that reach the library."""

import pytest

torch = pytest.importorskip("torch")

from int4_quantized_moe_amd import device, workloads  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The library is never reached, and CPU tensors pass for ones on a GPU that is not the current one."""
    seen, current = [], []

    class Current:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *a):
            current.pop()

    monkeypatch.setattr(device, "_gpu", lambda t: t.device)
    monkeypatch.setattr(device, "_elsewhere", lambda d: not current)
    monkeypatch.setattr(device, "_handle", lambda stream, dev: ("stream of", stream))
    monkeypatch.setattr(device, "_empty", lambda shape, dtype, dev, stream: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "device", Current)
    for name in ("kt_norm_fwd", "kt_norm_bwd", "kt_adamw_step", "kt_moe_decode"):
        monkeypatch.setattr(device._lib, name, lambda *a, name=name: seen.append((name, list(current), a)))
    return seen


def _only(calls, name, stream):
    (got, current, args), = calls
    assert got == name and current == [torch.device("cpu")] and args[-1] == ("stream of", stream)
    return args


@pytest.mark.parametrize("stream", [None, 5])
def test_norm(calls, stream):
    norm = device.DeviceNorm(8, weight=torch.ones(8))
    x, b = torch.zeros(3, 8), torch.zeros(3, 8, dtype=BF16)
    h, y = norm.forward(x, branch=b, stream=stream)
    args = _only(calls, "kt_norm_fwd", stream)
    assert args[1] == 3 and args[2] is x and args[3] is b and args[5] is h and args[6] is y and h.dtype is x.dtype and y.dtype is BF16
    calls.clear()
    ws, grads = norm.workspace(3, device="cpu"), norm.grad_buffers(fill=0.0)
    gx, gb = norm.backward(h, ws, grads, branch=b, grad_y=y, accumulate=True, grad_scale=0.5, stream=stream)
    args = _only(calls, "kt_norm_bwd", stream)
    assert args[2] is h and args[6] is y and args[7] is gx and args[8] is gb and args[10] is grads["weight"]
    assert args[15:18] == (True, 0.5, ws)


def test_norm_without_a_branch_or_outputs(calls):
    norm = device.DeviceNorm(8)
    x = torch.zeros(2, 8, dtype=BF16)
    h, y = norm.forward(x)
    assert h is x and y.shape == (2, 8)
    calls.clear()
    assert norm.backward(x, None, {}, grad_y=y, need_input=False) == (None, None)
    assert calls[0][2][7] is None and calls[0][2][8] is None


@pytest.mark.parametrize("stream", [None, 7])
def test_adamw(calls, stream):
    p = {"a": torch.zeros(3, 4), "b": torch.zeros(5, dtype=BF16)}
    opt = device.DeviceAdamW(p, master=True, max_norm=1.0, no_decay=("b",))
    grads = {"b": torch.ones(5, dtype=BF16), "a": torch.ones(3, 4), "more": torch.ones(1)}
    opt.step(grads, grad_scale=0.25, stream=stream)
    args = _only(calls, "kt_adamw_step", stream)
    hyper, tensors, count, step, norm, lr, ws = args[:7]
    assert count == 2 and step is opt.step_count and norm is opt.grad_norm and lr is None and ws is opt._workspace
    assert hyper.grad_scale == 0.25 and hyper.max_norm == 1.0
    assert [t.count for t in tensors] == [12, 5] and [t.decay for t in tensors] == [1, 0]
    assert [t.grad for t in tensors] == [grads[n].data_ptr() for n in "ab"]
    assert tensors[0].master is None and tensors[1].master == opt.state["b"]["master"].data_ptr()
    # another step's gradients take these ones' place
    calls.clear()
    grads["a"] = torch.ones(3, 4, dtype=BF16)
    opt.step(grads, lr=torch.ones(1), stream=stream)
    assert calls[0][2][1][0].grad == grads["a"].data_ptr() and calls[0][2][1][0].grad_type == device._lib.KT_TYPE_BF16


@pytest.mark.parametrize("wrong,word", [({"a": torch.ones(4, 3)}, "shape"), ({"a": torch.ones(4, 3).t()}, "contiguous"),
                                        ({"a": torch.ones(3, 4, dtype=torch.float64)}, "float32 or"), ({}, "no 'a'"),
                                        ({"a": torch.ones(3, 4, device="meta")}, "must be on")])
def test_adamw_refuses_a_step_s_gradients(calls, wrong, word):
    opt = device.DeviceAdamW({"a": torch.zeros(3, 4)})
    with pytest.raises(ValueError, match=word):
        opt.step(wrong)
    assert not calls


@pytest.mark.parametrize("stream", [None, 9])
def test_decode(calls, stream):
    layer = object.__new__(device.DeviceLayer)
    layer.cfg = workloads.LayerConfig("small", 8, 2, 64, 32, 4, 8.0, 5, 2.0)
    layer.device, layer.layer, layer.gate_packed = torch.device("cpu"), None, torch.zeros(1)
    x, ids, rw, ws = torch.zeros(3, 64, dtype=BF16), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2), torch.zeros(1, dtype=torch.uint8)
    out = layer.decode(x, ids, rw, ws, stream=stream)
    args = _only(calls, "kt_moe_decode", stream)
    assert args[1] == 3 and args[2] is x and args[3] is ids and args[4] is rw and args[5] is out and args[6] is ws
    assert out.shape == (3, 64) and out.dtype is BF16
