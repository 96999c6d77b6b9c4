"""GPU: the operators around the experts write nothing outside their outputs
and workspaces, one workspace serves every shorter batch, checkpoints of tensors large
enough for the form with four units a thread, and long batches through long
contractions.  Each case prints its name first."""

import math

import numpy as np
import pytest

from tests import block_reference as R
from tests.test_canaries import Guarded

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


class Buffers:
    """Guarded tensors by name."""

    def __init__(self):
        self.all = {}

    def new(self, name, shape, dtype):
        self.all[name] = b = Guarded(int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size())
        return b.view(dtype, shape)

    def check(self):
        torch.cuda.synchronize()
        broken = [n for n, b in self.all.items() if not b.intact()]
        assert not broken, f"guard bytes changed around {broken}"


# few tokens, splits with their partial sums, both tiles, odd widths
@pytest.mark.parametrize("t,k,n", [(3, 72, 5), (33, 7168, 100), (130, 136, 129), (300, 512, 384), (3471, 3656, 75),
                                   (75, 3656, 3471)])
@pytest.mark.parametrize("act,dtype,fmt", [("none", BF16, None), ("none", F32, "e4m3"), ("silu", F32, "int8")])
def test_dense_products_keep_to_their_buffers(dev, t, k, n, act, dtype, fmt):
    _say("dense", t, k, n, act, dtype, fmt)
    x, w, dy = _rand(1, t, k), _rand(2, n, k, std=k**-0.5), _rand(3, t, n, dtype=dtype)
    lin = dev.DeviceLinear(w, _rand(4, n, dtype=F32), act)
    b = Buffers()
    ws = b.new("workspace", (lin.workspace(t).numel(),), torch.uint8)
    wb = b.new("backward workspace", (lin.backward_workspace(t, checkpoint=fmt is not None).numel(),), torch.uint8)
    y, z = b.new("output", (t, n), dtype), b.new("preact", (t, n), BF16)
    dx = b.new("grad_input", (t, k), BF16)
    grads = {"weight": b.new("d_weight", (n, k), F32), "bias": b.new("d_bias", (n,), F32)}
    lin.forward(x, ws, residual=_rand(5, t, n), preact=z, output=y)
    kept = x if fmt is None else dev.pack_checkpoint8(x, fmt)
    lin.backward(kept, dy, wb, grads, preact=z, grad_input=dx, grad_residual=x)
    b.check()


@pytest.mark.parametrize("t,e,k,groups", [(1, 384, 8, 8), (33, 60, 4, 4), (300, 384, 8, 1), (7, 1000, 20, 4), (19, 513, 9, 1)])
@pytest.mark.parametrize("score,dtype", [("softmax", BF16), ("sigmoid", F32)])
def test_routing_keeps_to_its_buffers(dev, t, e, k, groups, score, dtype):
    _say("routing", t, e, k, groups, score, dtype)
    b = Buffers()
    logits = _rand(1, t, e, dtype=dtype)
    router = dev.DeviceRouter(e, k, score=score, num_groups=groups, top_groups=max(1, groups // 2),
                              bias=b.new("bias", (e,), F32).zero_())
    ids, w = b.new("ids", (t, k), torch.int64), b.new("weights", (t, k), F32)
    load = b.new("load", (e,), torch.int32)
    router.forward(logits, expert_ids=ids, route_weights=w, load=load)
    router.backward(logits, ids, _rand(2, t, k, dtype=F32), grad_logits=b.new("grad_logits", (t, e), dtype))
    router.update_bias(load, 0.125)
    b.check()


@pytest.mark.parametrize("rows,cols", [(4693, 7168), (32771, 1000)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_checkpoints_of_large_tensors(dev, rows, cols, fmt):
    """From 2^21 half groups a thread takes four of them; the same rows in pieces below that give the same bytes
    (whose values the small cases check)."""
    _say("large checkpoint", rows, cols, fmt)
    groups = -(-cols // 32)
    assert rows * groups * 2 >= 2**21 and rows * groups * 2 % 1024
    x = _rand(rows, rows, cols) * torch.exp(_rand(1, cols))
    x[rows - 1, cols - 1] = float("inf")
    b = Buffers()
    ck = dev.Checkpoint8(b.new("codes", (rows, cols), torch.int8), b.new("scales", (rows, groups), torch.uint8), fmt)
    out = b.new("rows", (rows, cols), BF16)
    dev.pack_checkpoint8(x, fmt, ck)
    dev.unpack_checkpoint8(ck, out)
    b.check()
    step = 1024
    assert step * groups * 2 < 2**21
    for at in range(0, rows, step):
        part = dev.pack_checkpoint8(x[at:at + step], fmt)
        assert torch.equal(part.codes, ck.codes[at:at + step]) and torch.equal(part.scales, ck.scales[at:at + step])
        back = dev.unpack_checkpoint8(part)
        assert torch.equal(back.view(torch.int16), out[at:at + step].view(torch.int16))


@pytest.mark.parametrize("t,k,n", [(4096, 7168, 384), (3001, 7168, 2048), (1536, 2048, 7168)])
def test_long_batches_through_long_contractions(dev, t, k, n):
    """Both products and all gradients, in 64 bits on the GPU; bounds as in block_reference, with three planes of dz
    for the weight and half a step of what bf16 leaves of dz (2^-16) for the input."""
    _say("long", t, k, n)
    x, w, dy = _rand(1, t, k), _rand(2, n, k, std=k**-0.5), _rand(3, t, n, dtype=F32)
    xd, wd, dz = x.double(), w.double(), dy.double()
    lin = dev.DeviceLinear(w)
    y = lin.forward(x, lin.workspace(t), dtype=F32)
    R.within("y", y, xd @ wd.t(), 8 * math.sqrt(k) * R.U * (xd.abs() @ wd.abs().t()))
    grads = lin.grad_buffers()
    dx = lin.backward(x, dy, lin.backward_workspace(t), grads)
    want = dz @ wd
    bound = (2.0**-16 + 8 * math.sqrt(2 * n) * R.U) * (dz.abs() @ wd.abs())
    R.within("dx", dx, want, bound + R.UB * want.abs())
    R.within("dw", grads["weight"], dz.t() @ xd, (8 * math.sqrt(3 * t) + 1) * R.U * (dz.abs().t() @ xd.abs()))


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
