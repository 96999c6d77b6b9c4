"""GPU: dense products with their epilogue and gradients, against plain 64-bit
products within the bounds derived in block_reference.  Each case prints its
name first."""

import math

import pytest

from tests import block_reference as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[linear]", *a, flush=True)


def _rand(seed, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


SHAPES = [
    (1, 8, 1), (1, 7168, 384), (2, 72, 3), (3, 256, 17), (15, 136, 33), (16, 512, 64), (17, 64, 100), (31, 1024, 384),
    (33, 200, 65), (64, 128, 128), (65, 264, 130), (100, 512, 8), (127, 96, 250), (128, 2048, 256), (200, 72, 6),
    (257, 320, 129), (300, 512, 384), (513, 1000, 257), (1025, 128, 520), (2049, 64, 24),
]


def _forward(dev, t, k, n, act, bias, residual, preact, dtype, seed=0):
    x, w = _rand(seed + 1, t, k), _rand(seed + 2, n, k, std=k**-0.5)
    b = _rand(seed + 3, n, dtype=F32) if bias else None
    r = _rand(seed + 4, t, n) if residual else None
    lin = dev.DeviceLinear(w, b, act)
    z = torch.full((t, n), 7.0, dtype=BF16, device="cuda") if preact else None
    ws = lin.workspace(t)
    ws.fill_(0xFF)
    out = torch.full((t, n), 7.0, dtype=dtype, device="cuda")
    lin.forward(x, ws, residual=r, preact=z, output=out)
    y, zr, yb, zb = R.linear(x, w, b, r, act)
    R.within("y", out, y, yb + R.rounding(dtype) * y.abs())
    if preact:
        R.within("z", z, zr, zb + R.UB * zr.abs())


@pytest.mark.parametrize("t,k,n", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_shapes(dev, t, k, n, dtype):
    _say("forward", t, k, n, dtype)
    _forward(dev, t, k, n, "none", False, False, False, dtype)
    _forward(dev, t, k, n, "silu", True, True, True, dtype, seed=10)


@pytest.mark.parametrize("t,k,n", [(3471, 136, 3613), (6200, 8, 2056), (3471, 200, 3656)])
def test_forward_large_tiles(dev, t, k, n):
    """Shapes that the 256 x 256 tiles take, ragged in every direction."""
    _say("large", t, k, n)
    _forward(dev, t, k, n, "none", False, False, False, F32)
    _forward(dev, t, k, n, "gelu", True, True, True, BF16, seed=10)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual,preact", [(0, 0, 0), (1, 0, 1), (0, 1, 0), (1, 1, 1)])
@pytest.mark.parametrize("t,k,n", [(5, 512, 40), (130, 136, 129), (300, 256, 260)])
def test_forward_epilogues(dev, act, bias, residual, preact, t, k, n):
    _say("epilogue", act, bias, residual, preact, t, k, n)
    for dtype in (BF16, F32):
        _forward(dev, t, k, n, act, bias, residual, preact, dtype)


def test_forward_in_place_residual(dev):
    _say("in place")
    for t in (3, 200):
        x, w = _rand(1, t, 96), _rand(2, 72, 96, std=0.1)
        y = _rand(3, t, 72)
        before = y.clone()
        lin = dev.DeviceLinear(w, None, "relu")
        lin.forward(x, lin.workspace(t), residual=y, output=y)
        want, _, b, _ = R.linear(x, w, None, before, "relu")
        R.within("in place", y, want, b + R.UB * want.abs())


def test_outputs_keep_their_neighbours(dev):
    """Nothing is written outside the outputs (rows behind the last token, columns of odd widths)."""
    _say("neighbours")
    for t, k, n in ((1, 64, 3), (5, 64, 7), (130, 64, 129), (33, 72, 384)):
        for dtype in (BF16, F32):
            flat = torch.full((t * n + 64,), 5.0, dtype=dtype, device="cuda")
            x, w = _rand(1, t, k), _rand(2, n, k)
            lin = dev.DeviceLinear(w)
            out = flat[32:32 + t * n].view(t, n)
            lin.forward(x, lin.workspace(t), output=out)
            assert (flat[:32] == 5).all() and (flat[32 + t * n:] == 5).all()
            want, _, b, _ = R.linear(x, w)
            R.within("neighbours", out, want, b + R.rounding(dtype) * want.abs())
        gw = torch.full((n * k + 64,), 5.0, device="cuda")
        gx = torch.full((t * k + 64,), 5.0, dtype=BF16, device="cuda")
        dy = _rand(3, t, n)
        lin.backward(x, dy, lin.backward_workspace(t), {"weight": gw[32:32 + n * k].view(n, k)},
                     grad_input=gx[32:32 + t * k].view(t, k))
        for f, m in ((gw, n * k), (gx, t * k)):
            assert (f[:32] == 5).all() and (f[32 + m:] == 5).all()


def test_not_finite_inputs_stay_in_their_rows_and_columns(dev):
    _say("not finite")
    for t, k, n in ((9, 64, 40), (200, 264, 130)):
        x, w = _rand(1, t, k), _rand(2, n, k)
        x[3, 7] = float("nan")
        x[5, 60] = float("inf")
        w[11, 9] = float("nan")
        lin = dev.DeviceLinear(w)
        y = lin.forward(x, lin.workspace(t), dtype=F32).cpu()
        nan = torch.isnan(y)
        want = torch.zeros_like(nan)
        want[3] = True
        want[:, 11] = True
        assert torch.equal(nan, want)
        rest = torch.isinf(y)
        assert bool(rest[5, :11].all()) and int(rest.sum()) == n - 1


@pytest.mark.parametrize("act", ACTS[1:])
def test_extreme_preactivations(dev, act):
    """Values at which a formula's parts overflow: the results are those of the limits."""
    _say("extremes", act)
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 20.0, -20.0, 88.0, -88.0, 1e4, -1e4, 1e20, -1e20, 3e38,
                      -3e38], dtype=F32)
    x = torch.zeros(16, 16, dtype=BF16, device="cuda")
    x[:, 0] = v.to(BF16).cuda()
    w = torch.zeros(8, 16, dtype=BF16, device="cuda")
    w[:, 0] = 1
    lin = dev.DeviceLinear(w, None, act)
    z = torch.empty(16, 8, dtype=BF16, device="cuda")
    y = lin.forward(x, lin.workspace(16), preact=z, dtype=F32)
    zd = v.to(BF16).double()
    lim = zd.clamp(-40, 40)  # the limits are reached there, in 64 bits too
    want = torch.where(zd < -40, 0.0, torch.where(zd > 40, zd, R.act(lim, act)))
    R.within("value", y[:, 3], want, 1e-6 * want.abs() + 1e-7)
    grads = lin.grad_buffers()
    dx = lin.backward(x, torch.ones(16, 8, dtype=BF16, device="cuda"), lin.backward_workspace(16), grads, preact=z)
    slope = torch.where(zd < -40, 0.0, torch.where(zd > 40, 1.0, R.act_grad(lim, act)))
    R.within("slope", dx[:, 0], 8 * slope, 2 * R.UB * (8 * slope).abs() + 1e-5)


def test_gelu_keeps_the_digits_of_its_tail(dev):
    """z Phi(z) and its slope for z far below 0, relative to their own size.  erfc is within 16 units of
    its last place (2^-23), and its argument u = z / sqrt(2) within two roundings, which it magnifies by 2 u^2 + 1;
    the slope's exponential magnifies z^2 / 2's three roundings by z^2 / 2."""
    _say("gelu's tail")
    v = torch.tensor([-0.5, -1, -2, -3, -4, -5, -6, -7, -8, -9, -10, -10.5, -11, -11.5, -11.75, -12], dtype=F32)
    x = torch.zeros(16, 16, dtype=BF16, device="cuda")
    x[:, 0] = v.to(BF16).cuda()
    w = torch.zeros(8, 16, dtype=BF16, device="cuda")
    w[:, 0] = 1
    lin = dev.DeviceLinear(w, None, "gelu")
    z = torch.empty(16, 8, dtype=BF16, device="cuda")
    y = lin.forward(x, lin.workspace(16), preact=z, dtype=F32)
    zd = v.double()
    want = R.act(zd, "gelu")
    rel = 16 * 2.0**-23 + (zd * zd + 1) * 2.0**-23 + 4 * R.U
    R.within("value", y[:, 3], want, rel * want.abs())
    dx = lin.backward(x, torch.ones(16, 8, dtype=BF16, device="cuda"), lin.backward_workspace(16), {}, preact=z)
    slope = R.act_grad(zd, "gelu")
    parts = R.act(zd, "gelu").abs() / zd.abs() + zd.abs() * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    R.within("slope", dx[:, 0], 8 * slope, 8 * (2.01 * R.UB * slope.abs() + (rel + 3 * zd * zd * R.U) * parts))


@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_of_minus_infinity(dev, act):
    """Their limit there is 0, and so is their slope's."""
    _say("minus infinity", act)
    for t in (3, 200):
        x = torch.zeros(t, 16, dtype=BF16, device="cuda")
        x[:, 0] = -float("inf")
        w = torch.zeros(8, 16, dtype=BF16, device="cuda")
        w[:, 0] = 1
        lin = dev.DeviceLinear(w, None, act)
        z = torch.empty(t, 8, dtype=BF16, device="cuda")
        y = lin.forward(x, lin.workspace(t), preact=z, dtype=F32)
        assert torch.isneginf(z).all() and (y == 0).all()
        dx = lin.backward(x, torch.ones(t, 8, dtype=BF16, device="cuda"), lin.backward_workspace(t), {}, preact=z)
        assert (dx == 0).all()


# ---------------------------------------------------------------- gradients


def _backward(dev, t, k, n, act, dtype, residual=False, ckpt=None, accumulate=False, scale=1.0, bias=True, seed=0):
    x, w = _rand(seed + 1, t, k), _rand(seed + 2, n, k, std=n**-0.5)
    b = _rand(seed + 3, n, dtype=F32) if bias else None
    dy = _rand(seed + 4, t, n, dtype=dtype)
    z = _rand(seed + 5, t, n) if act != "none" else None
    r = _rand(seed + 6, t, k) if residual else None
    lin = dev.DeviceLinear(w, b, act)
    ws = lin.backward_workspace(t, checkpoint=ckpt is not None)
    ws.fill_(0xFF)
    grads = lin.grad_buffers(fill=0.75)
    dx = torch.full((t, k), 7.0, dtype=BF16, device="cuda")
    kept = x
    if ckpt:
        kept = dev.pack_checkpoint8(x, ckpt)
        x = dev.unpack_checkpoint8(kept)
    lin.backward(kept, dy, ws, grads, preact=z, grad_input=dx, grad_residual=r, accumulate=accumulate,
                 grad_scale=scale)
    want, bound = R.linear_bwd(x, w, dy, z, r, act)
    R.within("dx", dx, want["dx"], bound["dx"] + R.UB * want["dx"].abs())
    base = 0.75 if accumulate else 0.0
    for name, key in (("weight", "dw"), ("bias", "db")):
        if name in grads:
            e = base + scale * want[key]
            R.within(key, grads[name], e, abs(scale) * bound[key] + 2 * R.U * (e.abs() + base))


@pytest.mark.parametrize("t,k,n", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_shapes(dev, t, k, n, dtype):
    _say("backward", t, k, n, dtype)
    _backward(dev, t, k, n, "none", dtype, bias=False)
    _backward(dev, t, k, n, "silu", dtype, residual=True, seed=20)


@pytest.mark.parametrize("t,k,n", [(3471, 3656, 75), (75, 3656, 3471), (130, 3656, 3472)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_large_tiles(dev, t, k, n, dtype):
    """Shapes whose grad_input or weight gradient the 256 x 256 tiles take."""
    _say("large backward", t, k, n, dtype)
    _backward(dev, t, k, n, "none", dtype, accumulate=True, scale=0.5)
    _backward(dev, t, k, n, "silu", dtype, residual=True, ckpt="int8", seed=20)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,k,n", [(7, 256, 40), (130, 136, 129), (520, 264, 72)])
def test_backward_forms(dev, act, dtype, t, k, n):
    _say("forms", act, dtype, t, k, n)
    _backward(dev, t, k, n, act, dtype, residual=True, accumulate=True, scale=0.25)
    _backward(dev, t, k, n, act, dtype, ckpt="int8")
    _backward(dev, t, k, n, act, dtype, ckpt="e4m3", accumulate=True, scale=-2.0)


def test_backward_parts_alone(dev):
    """Each gradient alone gives what all together give, bit for bit; grad_input in place of the residual."""
    _say("parts")
    for t, k, n, act, dtype in ((40, 64, 24, "gelu", BF16), (300, 136, 130, "none", F32), (33, 64, 7, "none", BF16)):
        x, w, dy = _rand(1, t, k), _rand(2, n, k), _rand(3, t, n, dtype=dtype)
        z = _rand(4, t, n) if act != "none" else None
        r = _rand(5, t, k)
        lin = dev.DeviceLinear(w, _rand(6, n, dtype=F32), act)
        ws = lin.backward_workspace(t)
        all_g = lin.grad_buffers()
        dx = lin.backward(x, dy, ws, all_g, preact=z, grad_residual=r)
        inplace = r.clone()
        assert lin.backward(x, dy, ws, {}, preact=z, grad_residual=inplace, grad_input=inplace) is inplace
        assert torch.equal(inplace, dx)
        for name in ("weight", "bias"):
            one = {name: torch.full_like(all_g[name], 3.0)}
            assert lin.backward(x, dy, ws, one, preact=z, need_input=False) is None
            assert torch.equal(one[name], all_g[name])


def test_backward_without_tokens(dev):
    _say("no tokens")
    lin = dev.DeviceLinear(_rand(1, 24, 64), _rand(2, 24, dtype=F32))
    x, dy = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 24, dtype=BF16, device="cuda")
    assert lin.forward(x, lin.workspace(0)).shape == (0, 24)
    grads = lin.grad_buffers(fill=2.0)
    lin.backward(x, dy, lin.backward_workspace(0), grads, accumulate=True)
    assert (grads["weight"] == 2).all() and (grads["bias"] == 2).all()
    lin.backward(x, dy, lin.backward_workspace(0), grads)
    assert not grads["weight"].any() and not grads["bias"].any()


def test_backward_of_not_finite_gradients(dev):
    """An infinite or NaN grad_output reaches the gradients of its row and column alone; fp32 values above
    bf16's largest number stay finite in the weight's gradient."""
    _say("not finite gradients")
    t, k, n = 40, 64, 24
    x, w = _rand(1, t, k), _rand(2, n, k)
    x[:, 0] = 0.0
    x[3, 0] = 2.0**-20
    dy = _rand(3, t, n, dtype=F32)
    dy[3, 5] = 3.4e38  # rounds to infinity in bf16
    lin = dev.DeviceLinear(w)
    grads = lin.grad_buffers()
    lin.backward(x, dy, lin.backward_workspace(t), grads, need_input=False)
    assert torch.isfinite(grads["weight"][5, 0]) and torch.isfinite(grads["weight"][:5]).all()
    want = 3.4e38 * 2.0**-20
    assert abs(float(grads["weight"][5, 0]) - want) <= 2.0**-16 * want
    dy[3, 5] = float("inf")
    x[3] = x[3].abs() + 0.5
    dx = lin.backward(x, dy, lin.backward_workspace(t), grads)
    assert torch.isinf(grads["weight"][5]).all() and torch.isfinite(grads["weight"][:5]).all()
    assert not torch.isfinite(dx[3]).any() and torch.isfinite(dx[:3]).all() and torch.isfinite(dx[4:]).all()


def test_results_are_the_same_every_time(dev):
    _say("determinism")
    for t, k, n in ((1, 512, 384), (40, 7168, 384), (600, 512, 130)):
        x, w, dy = _rand(1, t, k), _rand(2, n, k), _rand(3, t, n, dtype=F32)
        lin = dev.DeviceLinear(w, _rand(4, n, dtype=F32))
        runs = []
        for fill in (0xFF, 0x11, 0x00):
            ws, wb, g = lin.workspace(t), lin.backward_workspace(t), lin.grad_buffers()
            ws.fill_(fill)
            wb.fill_(fill)
            y = lin.forward(x, ws)
            runs.append((y, lin.backward(x, dy, wb, g), g["weight"], g["bias"]))
        for other in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
