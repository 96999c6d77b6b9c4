"""The operators around the experts on the CPU: a workspace sized for the longest
batch serves every shorter one, and the experts' backward from a checkpoint
checks what it writes to."""

import pytest

import int4_quantized_moe_amd as kt

torch = pytest.importorskip("torch")
from int4_quantized_moe_amd import device, workloads  # noqa: E402

FAKE = 1 << 20  # a non-null, 256-aligned address; never dereferenced by the size functions


@pytest.mark.parametrize("k,n", [(64, 24), (512, 384), (1024, 1), (2048, 2048), (7168, 384), (7168, 2048), (2048, 7168),
                                 (65536, 8), (8, 65536)])
@pytest.mark.parametrize("act", [0, 2])
def test_workspaces_grow_with_the_tokens(k, n, act):
    lin = kt.kt_linear(k, n, act, FAKE, None)
    tokens = [*range(0, 400), *range(400, 9000, 61), *(128 * r for r in range(1, 160)), *(128 * r + 1 for r in range(1, 160)),
              1 << 15, 1 << 18, 1 << 20]
    last = [0, 0, 0]
    for t in sorted(set(tokens)):
        sizes = [kt.kt_linear_workspace_bytes(lin, t), kt.kt_linear_bwd_workspace_bytes(lin, t),
                 kt.kt_linear_bwd_workspace_bytes(lin, t, True)]
        assert all(a >= b for a, b in zip(sizes, last)), (t, sizes, last)
        last = sizes


# ---------------------------------------------------------------- the experts' backward from a checkpoint


def _checkpoint_call(monkeypatch):
    """A layer, its arguments and grads that the class takes for ones on a GPU; the library is never reached."""
    layer = object.__new__(device.DeviceLayer)
    layer.cfg = workloads.LayerConfig("small", 8, 2, 64, 32, 4, 8.0, 5, 2.0)
    layer.device, layer.layer, layer.gate_packed = torch.device("cpu"), None, torch.zeros(1)
    monkeypatch.setattr(device, "_gpu", lambda t: t.device)
    monkeypatch.setattr(device, "_elsewhere", lambda d: False)
    reached = []
    monkeypatch.setattr(device._lib, "kt_moe_bwd_ckpt8", lambda *a: reached.append(a))
    t = 5
    ck = device.Checkpoint8(torch.zeros(t, 64, dtype=torch.int8), torch.zeros(t, 2, dtype=torch.uint8), "int8")
    args = (ck, torch.zeros(t, 2, dtype=torch.int64), torch.zeros(t, 2), torch.zeros(t, 64, dtype=torch.bfloat16),
            torch.zeros(1, dtype=torch.uint8))
    return layer, args, layer.grad_buffers(fill=0.0), reached


def test_layer_class_checks_the_gradients_of_a_checkpoint_call(monkeypatch):
    layer, args, grads, reached = _checkpoint_call(monkeypatch)
    layer.backward(*args, grads)
    assert len(reached) == 1
    for name, g in grads.items():
        for wrong, word in ((g[:-1], name), (g.double(), name), (g.transpose(1, 2), name), (g.to("meta"), name)):
            with pytest.raises(ValueError, match=word):
                layer.backward(*args, {**grads, name: wrong})
        with pytest.raises(ValueError, match=name):
            layer.backward(*args, {n: v for n, v in grads.items() if n != name})
    layer.gate_packed = layer.gate_packed.to("meta")  # the layer's weights are elsewhere
    with pytest.raises(ValueError, match="checkpoint must be on"):
        layer.backward(*args, grads)
    assert len(reached) == 1


def test_layer_class_makes_the_checkpoint_s_gpu_current(monkeypatch):
    layer, args, grads, reached = _checkpoint_call(monkeypatch)
    current = []

    class Current:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *a):
            current.append(None)

    monkeypatch.setattr(device, "_elsewhere", lambda d: not current)
    monkeypatch.setattr(torch.cuda, "device", Current)
    dx, _ = layer.backward(*args, grads)
    assert current == [torch.device("cpu"), None] and len(reached) == 1 and dx.shape == (5, 64)
