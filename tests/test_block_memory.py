"""GPU: the workspaces of the operators around the experts.  Each case prints
its name first."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[block memory]", *a, flush=True)


def _rand(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("k,n,longest", [(7168, 384, 16384), (2048, 2048, 4096), (7168, 2048, 1024)])
def test_one_workspace_serves_shorter_batches(dev, k, n, longest):
    _say("one workspace", k, n, longest)
    w = _rand(2, n, k, std=k**-0.5)
    lin = dev.DeviceLinear(w)
    ws, wb = lin.workspace(longest), lin.backward_workspace(longest)
    for t in (1, 17, 64, 65, 129, 512, 1000, longest // 2 + 1, longest):
        x, dy = _rand(t, t, k), _rand(t + 1, t, n, dtype=F32)
        own, one = lin.grad_buffers(), lin.grad_buffers()
        a = lin.forward(x, lin.workspace(t)), lin.backward(x, dy, lin.backward_workspace(t), own)
        b = lin.forward(x, ws), lin.backward(x, dy, wb, one)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(own["weight"], one["weight"])
