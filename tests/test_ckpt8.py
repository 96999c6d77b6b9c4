"""GPU: 8-bit activation checkpoints, against a plain 64-bit implementation
(equal values), and the experts' backward from one (equal to the recompute
backward on the unpacked rows, bit for bit).  Each case prints its name."""

import numpy as np
import pytest

from int4_quantized_moe_amd import workloads as W
from tests import block_reference as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[ckpt8]", *a, flush=True)


def _round_trip(dev, x, fmt):
    ck = dev.checkpoint8_buffers(*x.shape, fmt)
    ck.codes.fill_(0x55)
    ck.scales.fill_(0x55)
    dev.pack_checkpoint8(x.cuda(), fmt, ck)
    out = torch.full(x.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    dev.unpack_checkpoint8(ck, out)
    return ck, out


def _check(dev, x, fmt):
    ck, out = _round_trip(dev, x, fmt)
    want = R.checkpoint(x.float().numpy(), fmt)
    R.within(f"{fmt} {tuple(x.shape)}", out, want, np.zeros(x.shape))
    # the codes are what the header says they are
    codes = ck.codes.cpu()
    v = codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    scale = np.repeat(ck.scales.cpu().numpy().astype(np.int32), 32, 1)[:, :x.shape[1]]
    fine = scale != 255
    assert np.array_equal(np.ldexp(v.double().numpy(), scale - 127)[fine], want[fine])
    assert np.array_equal(~fine, np.isnan(want)) and not codes.numpy()[~fine].any()


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 100), (4, 256), (33, 96),
                                       (17, 7168), (300, 40), (65, 1000), (129, 512), (3, 8192)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_round_trip(dev, rows, cols, fmt):
    _say(rows, cols, fmt)
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g))
    _check(dev, x.to(torch.bfloat16), fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_every_bf16_value(dev, fmt):
    """Each of the 65536 bit patterns alone in a group, and beside the group maxima on both sides of the borders."""
    _say("all values", fmt)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(2048, 1024, dtype=torch.bfloat16)
    x.view(-1)[torch.arange(65536) * 32 + torch.arange(65536) % 32] = bits
    _check(dev, x, fmt)
    for top in (1.0, 1.75, 1.765625, 1.984375, 1.9921875):  # the last three: 7 bits after the point
        y = torch.zeros(64, 32 * 20, dtype=torch.bfloat16)
        frac = torch.arange(64 * 600).float() / (64 * 600)
        y.view(64, 20, 32)[:, :, 1:31] = (frac * top).to(torch.bfloat16).view(64, 20, 30)
        y.view(64, 20, 32)[:, :, 0] = top
        _check(dev, y, fmt)
        _check(dev, (y.float() * 2.0**-126).to(torch.bfloat16), fmt)
        _check(dev, (y.float() * 2.0**126).to(torch.bfloat16), fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("cols", [64, 70])
def test_not_finite_groups(dev, fmt, cols):
    _say("not finite", fmt, cols)
    x = torch.randn(6, cols, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[0, 5] = float("nan")
    x[1, 40] = float("inf")
    x[2, cols - 1] = float("-inf")
    x[3] = 0
    x[4] = -0.0
    _check(dev, x, fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_unaligned_buffers_and_neighbours(dev, fmt):
    """Codes and scales that start 4 bytes into an allocation; the bytes around them stay."""
    _say("offsets", fmt)
    for rows, cols in ((3, 64), (5, 70), (4, 256)):
        x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(cols)).to(torch.bfloat16)
        groups = -(-cols // 32)
        codes = torch.full((rows * cols + 8,), 0x33, dtype=torch.int8, device="cuda")
        scales = torch.full((rows * groups + 8,), 0x44, dtype=torch.uint8, device="cuda")
        ck = dev.Checkpoint8(codes[4:-4].view(rows, cols), scales[4:-4].view(rows, groups), fmt)
        dev.pack_checkpoint8(x.cuda(), fmt, ck)
        rest = torch.full((rows * cols + 16,), 2.0, dtype=torch.bfloat16, device="cuda")
        out = dev.unpack_checkpoint8(ck, rest[8:-8].view(rows, cols))
        R.within("offsets", out, R.checkpoint(x.float().numpy(), fmt), np.zeros(x.shape))
        assert (codes[:4] == 0x33).all() and (codes[-4:] == 0x33).all()
        assert (scales[:4] == 0x44).all() and (scales[-4:] == 0x44).all()
        assert (rest[:8] == 2).all() and (rest[-8:] == 2).all()


def test_empty(dev):
    _say("empty")
    for shape in ((0, 64), (3, 0)):
        ck = dev.pack_checkpoint8(torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
        assert dev.unpack_checkpoint8(ck).shape == shape


def _bits(t):
    return t.detach().contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16).cpu().numpy()


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_experts_backward_from_a_checkpoint(dev, index, fmt):
    cfg, weights, batch = W.make_workload(index)
    _say("experts", cfg.name, fmt)
    dl, db = dev.DeviceLayer(cfg, weights), dev.DeviceBatch(batch)
    ck = dev.pack_checkpoint8(db.inputs, fmt)
    rows = dev.unpack_checkpoint8(ck)
    results = []
    for x, ws in ((rows, dl.workspace(db.qlen)), (ck, dl.checkpoint_workspace(db.qlen))):
        ws.fill_(0xFF)
        grads = dl.grad_buffers(fill=0.5)
        dr = torch.empty(batch.expert_ids.shape, dtype=torch.float32, device="cuda")
        dx, _ = dl.backward(x, db.expert_ids, db.route_weights, db.grad_output, ws, grads, accumulate=True,
                            grad_scale=0.25, grad_route=dr, recompute=True)
        results.append({"dx": _bits(dx), "dr": _bits(dr), **{n: _bits(g) for n, g in grads.items()}})
    for n in results[0]:
        assert np.array_equal(results[0][n], results[1][n]), n
