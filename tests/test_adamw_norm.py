"""GPU: AdamW's check for finite gradients goes by the norm that the caller reads."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_a_norm_beyond_fp32_changes_nothing():
    """Finite gradients whose norm fp32 does not hold: grad_norm says infinity, and nothing else has changed.  A norm just below is a step."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    for max_norm in (None, 1.0):
        params = {"a": torch.ones(300, device="cuda"), "b": torch.ones(5, device="cuda")}
        opt = device.DeviceAdamW(params, max_norm=max_norm, check_finite=True)
        opt.step({"a": torch.zeros(300, device="cuda"), "b": torch.full((5,), 3e38, device="cuda")})
        assert float(opt.grad_norm) == float("inf") and int(opt.step_count) == 0
        assert all((p == 1).all() and not opt.state[n]["m"].any() and not opt.state[n]["v"].any() for n, p in params.items())
        opt.step({"a": torch.zeros(300, device="cuda"), "b": torch.full((5,), 1.5e38, device="cuda")})
        assert abs(float(opt.grad_norm) / (1.5e38 * 5**0.5) - 1) < 1e-6 and int(opt.step_count) == 1
