"""AdamW over more chunks than a launch takes: on the CPU how many that are, on the GPU that values behind
them are updated as they are alone."""

import os
import re

import pytest

from .conftest import ROOT

torch = pytest.importorskip("torch")

SOURCE = open(os.path.join(ROOT, "int4_quantized_moe_amd", "csrc", "kt_adamw.hip")).read()
CHUNK = 4 * 4 * 256  # values of a workgroup


def _launch():
    """Chunks that a launch of the update takes at most."""
    found = re.search(r"constexpr int64_t kAdamLaunch = 1 << (\d+)", SOURCE)
    return 1 << int(found.group(1)) if found else 2**36 // CHUNK * 32


def test_a_launch_stays_below_two_to_the_32_threads():
    """The header's largest tensors, 2^36 values each, have 2^24 chunks of 256 threads."""
    assert _launch() * 256 < 2**32


@pytest.mark.gpu
@pytest.mark.parametrize("states", ["fp32", "e4m3"])
def test_values_of_a_second_launch(states):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    print("[adamw launches]", states, flush=True)
    n, tail = _launch() * CHUNK + CHUNK * 2 + 77, CHUNK * 5 + 77
    make = lambda seed, *s: torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()  # noqa: E731
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:], g[-tail:] = make(1, tail), make(2, tail)
    rest, rest_grad = make(3, 5000), make(4, 5000)  # a tensor behind the large one
    alone = {"p": p[-tail:].clone(), "q": rest.clone()}
    big = device.DeviceAdamW({"p": p, "q": rest}, states=states, check_finite=True)
    small = device.DeviceAdamW(alone, states=states, check_finite=True)
    for _ in range(2):
        big.step({"p": g, "q": rest_grad})
        small.step({"p": g[-tail:].clone(), "q": rest_grad})
    assert torch.equal(p[-tail:], alone["p"]) and torch.equal(rest, alone["q"]) and not p[:-tail].any()
    assert torch.equal(big.grad_norm, small.grad_norm) and int(big.step_count) == 2
    for k in ("m", "v"):
        assert torch.equal(big.state["p"][k][-tail:].view(torch.uint8), small.state["p"][k].view(torch.uint8))
        assert torch.equal(big.state["q"][k].view(torch.uint8), small.state["q"][k].view(torch.uint8))
