"""GPU: the experts for a few tokens at the ends of their inputs' and scales' range: the largest inputs that their header allows,
subnormal ones, and what inputs that are not finite give in both formats.  Each case prints its name."""

import pytest

from tests import step_reference as S
from tests.test_decode import BF16, Case

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[decode range]", *a, flush=True)


# (2048 wide with 12288 slots x intermediate: the kernel of short rows; wider: the other)
SIZES = [(3, 4, 2, 128, 64), (3, 4, 2, 2080, 64), (8, 16, 2, 96, 1056)]


@pytest.mark.parametrize("t,e,k,h,i", SIZES)
@pytest.mark.parametrize("fmt", ["rawint4", "mxfp4"])
def test_the_largest_inputs(dev, t, e, k, h, i, fmt):
    """All inputs 2^120, of one sign and of random ones, under scales that bring the products back."""
    _say("largest", t, e, k, h, i, fmt)
    for signs in (False, True):
        c = Case(dev, t, e, k, h, i, 0, fmt, 1.0)
        c.x = torch.full_like(c.x, 2.0**120)
        if signs:
            c.x *= (torch.rand(t, h, device="cuda") < 0.5).to(BF16) * 2 - 1
        for n in ("gate_scale", "up_scale"):
            c.weights[n] *= 2.0**-122
        c.check(c.run())


@pytest.mark.parametrize("t,e,k,h,i", SIZES)
@pytest.mark.parametrize("fmt", ["rawint4", "mxfp4"])
def test_subnormal_inputs_and_scales(dev, t, e, k, h, i, fmt):
    """Inputs below 2^-126 (multiples of 2^-133: products with a code and their sums are exact in fp32) under large scales, and
    subnormal scales under large inputs."""
    _say("subnormal", t, e, k, h, i, fmt)
    c = Case(dev, t, e, k, h, i, 0, fmt)
    c.x = (torch.randint(-127, 128, (t, h), device="cuda").double() * 2.0**-133).to(BF16)
    assert float(c.x.double().abs().max()) < 2.0**-126 and c.x.double().any()
    for n in ("gate_scale", "up_scale"):
        c.weights[n] *= 2.0**126
    c.check(c.run())
    c = Case(dev, t, e, k, h, i, 0, fmt)
    c.x *= 2.0**100
    c.x *= 2.0**20
    for n in ("gate_scale", "up_scale"):  # from 2^-127 on: subnormal
        small = (torch.randint(1, 128, c.weights[n].shape, device="cuda").double() * 2.0**-133).to(BF16)
        c.weights[n].copy_(small if fmt == "rawint4" else torch.full_like(small, 2.0**-130))
    c.check(c.run())


@pytest.mark.parametrize("t,e,k,h,i", SIZES)
@pytest.mark.parametrize("limit", [0.0, 2.0])
def test_rawint4_inputs_that_are_not_finite(dev, t, e, k, h, i, limit):
    """They make their token's output NaN, clamped or not, and no other's; a token without an expert gets zeros whatever it holds."""
    _say("rawint4", t, e, k, h, i, limit)
    for value in (INF, -INF, NAN):
        c = Case(dev, t, e, k, h, i, 0, "rawint4", limit)
        want = c.run()
        c.x[1, h // 2] = value
        out = c.run()
        assert torch.isnan(out[1]).all()
        assert torch.equal(out[0], want[0]) and torch.equal(out[2:], want[2:])
        c.ids[1] = -1
        assert not c.run()[1].any()


@pytest.mark.parametrize("t,e,k,h,i", SIZES)
def test_mxfp4_inputs_that_are_not_finite(dev, t, e, k, h, i):
    """NaN makes its token's output NaN.  An infinite one goes by the formula: with weights of one sign its sums are infinite, which the clamp
    makes the limit; without the clamp the output is infinite, beside finite values of h whatever their size; an infinity times zero is NaN."""
    _say("mxfp4", t, e, k, h, i)
    for limit in (0.0, 2.0):
        c = Case(dev, t, e, k, h, i, 0, "mxfp4", limit)
        want = c.run()
        c.x[1, 5] = NAN
        out = c.run()
        assert torch.isnan(out[1]).all() and torch.equal(out[0], want[0]) and torch.equal(out[2:], want[2:])

        # the input's weights in gate and up are positive; all of down's are
        c = Case(dev, t, e, k, h, i, 0, "mxfp4", limit)
        for n in ("gate", "up"):
            c.weights[n + "_packed"][:, :, 0] = 0x33
        c.weights["down_packed"].copy_(c.weights["down_packed"] & 0x77 | 0x11)
        c.x[1, 0] = 2.0**110
        large = c.run()
        c.x[1, 0] = INF
        out = c.run()
        if limit:
            c.x[1, 0] = 2.0**110  # clamped to the same
            c.check(out)
            assert torch.equal(out, large)
        else:
            assert (out[1] == INF).all() and torch.equal(out[0], large[0]) and torch.equal(out[2:], large[2:])
    c = Case(dev, t, e, k, h, i, 0, "mxfp4")
    for n in ("gate", "up"):
        c.weights[n + "_packed"][:, :, 0] = 0x33
    c.weights["down_packed"][:] = 0x33
    c.weights["down_packed"][:, 1, i // 2 - 1] = 0x03  # a zero in the second row
    c.x[1, 0] = INF
    out = c.run()
    assert torch.isnan(out[1, 1]) and (out[1, 2:] == INF).all() and out[1, 0] == INF and torch.isfinite(out[0]).all()


def test_mxfp4_infinite_h_beside_finite_ones(dev):
    """One column of 16 of h is infinite, others are beyond fp16's range and have weights of the other sign: the output is infinite, not NaN."""
    _say("mxfp4 neighbours")
    c = Case(dev, 1, 1, 1, 32, 32, 0, "mxfp4")
    for n in ("gate", "up"):
        c.weights[n + "_packed"][:] = 0x22  # 1
        c.weights[n + "_scale"][:] = 1.0
    c.weights["gate_scale"][0, 3] = 2.0**60
    c.weights["up_scale"][0, 3] = 2.0**70
    c.weights["down_packed"][:] = 0xAA  # -1
    c.weights["down_packed"][:, :, 1] = 0x2A  # column 3: 1
    c.weights["down_scale"][:] = 1.0
    c.x[:] = 64.0
    out = c.run()
    want, _ = S.experts(c.x, c.ids, c.rw, c.weights, "mxfp4")
    assert float(want.min()) > 3.4e38  # beyond fp32: h of column 3 is infinite there
    assert (out == INF).all()
