"""GPU: the routing gradient and weights at the ends of the scores' range.  Each
case prints its name first."""

import numpy as np
import pytest

from tests import block_reference as R

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

STEP = 2.0**-149  # fp32's smallest number: a score below 2^-126 is held in steps of it


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[router extremes]", *a, flush=True)


def _slots(seed, t, e, k):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(t)])
    return ids, rng.standard_normal((t, k)).astype(np.float32)


def _gradient(dev, l, ids, g, **cfg):
    router = dev.DeviceRouter(l.shape[1], ids.shape[1], **cfg)
    out = torch.full(l.shape, 3.0, dtype=l.dtype, device="cuda")
    return router.backward(l.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(g).cuda(), grad_logits=out)


@pytest.mark.parametrize("e,k", [(384, 8), (600, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm,scale,size", [(True, 1e25, 1.0), (True, 3e38, 1.0), (False, 3e38, 100.0)])
def test_gradient_of_scores_that_vanish_under_a_large_scale(dev, e, k, score, renorm, scale, size):
    """Every chosen s is 0 in fp32, and so is its gradient, however large scale / 1e-20 and scale * g are.  (A softmax has
    one expert that holds all of it, chosen by nobody.)"""
    _say("vanished", e, k, score, renorm, scale)
    t = 37
    rng = np.random.default_rng(e)
    l = (rng.standard_normal((t, e)) - 300).astype(np.float32)
    ids, g = _slots(e + 1, t, e - 1, k)
    ids += 1
    if score == "softmax":
        l[:, 0] = 0.5
    for dtype in (torch.float32, torch.bfloat16):
        out = _gradient(dev, torch.from_numpy(l).to(dtype), ids, g * np.float32(size), score=score, renormalize=renorm,
                        scale=scale)
        # |dl| <= scale * |g| * e^-294 / 1e-20 < 1e-60
        assert (out == 0).all()
