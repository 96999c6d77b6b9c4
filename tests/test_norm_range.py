"""GPU: the norms over the range of values that their header gives, forward and backward.  Each case prints its name."""

import pytest

from tests import block_reference as R
from tests import step_reference as S
from tests.test_norm import BF16, F32, _make

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


@pytest.mark.parametrize("h", [7, 513, 7168, 16384])
@pytest.mark.parametrize("kind,stream", [("rms", F32), ("layer", BF16)])
@pytest.mark.parametrize("size", [2.0**56, 2.0**-50])
def test_values_at_the_ends_of_the_range(dev, h, kind, stream, size):
    """All values up to 2^56, or around 2^-50 with eps 0: their squares and sums stay in fp32."""
    print("[norm range]", h, kind, stream, size, flush=True)
    t = 5
    i, v, n = _make(h, t, h, F32, True, True, "channel", False)
    x = (torch.rand(t, h, generator=torch.Generator().manual_seed(h)) * 2 - 1).cuda()
    i["x"] = ((0.5 + 0.5 * x.abs()) * x.sign() * size).to(stream)
    i["branch"] = (i["branch"].float().clamp(-1, 1) * size).to(BF16)
    norm = dev.DeviceNorm(h, kind, eps=0.0, branch_norm=True, **v)
    hh, y = norm.forward(i["x"], branch=i["branch"])
    args = dict(kind=kind, eps=0.0, scale=1.0, branch_norm=True, **v)
    want_h, dh, want_y, dy = S.norm_fwd(i["x"], i["branch"], None, **args)
    R.within("h", hh, want_h, dh + S.rounding(stream) * (want_h.abs() + dh))
    R.within("y", y, want_y, dy + R.UB * (want_y.abs() + dy))
    gy = n(t, h).to(BF16).cuda()
    grads = norm.grad_buffers()
    gx, gb = norm.backward(hh, norm.workspace(t), grads, branch=i["branch"], grad_y=gy)
    want = S.norm_bwd(hh, i["branch"], None, None, gy, **args)
    for name, got, half in [("x", gx, S.rounding(stream)), ("branch", gb, R.UB)] + [(k, g, 2 * R.U) for k, g in grads.items()]:
        e, b = want[name]
        R.within(name, got, e, b + half * (e.abs() + b) + 2.0**-133)
