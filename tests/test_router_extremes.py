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


@pytest.mark.parametrize("e,k", [(384, 8), (40, 6), (700, 8), (384, 20)])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_of_large_logits(dev, e, k, renorm):
    """s (1 - s) keeps its digits where s is close to 1: each of the factors is within `prec` of its own size."""
    _say("large logits", e, k, renorm)
    t = 29
    rng = np.random.default_rng(e)
    l = np.where(rng.random((t, e)) < 0.7, rng.uniform(8, 80, (t, e)), rng.uniform(-20, 8, (t, e))).astype(np.float32)
    ids, g = _slots(e + 1, t, e, k)
    out = _gradient(dev, torch.from_numpy(l), ids, g, score="sigmoid", renormalize=renorm, scale=1.5)
    s = R.scores(l, "sigmoid")
    comp = 1.0 / (1.0 + np.exp(l.astype(np.float64)))  # 1 - s, which as a difference ends at l = 37 in 64 bits too
    si, g64 = np.take_along_axis(s, ids, 1), g.astype(np.float64)
    total = si.sum(1, keepdims=True) + 1e-20 if renorm else 1.0
    d = (g64 * si).sum(1, keepdims=True) / total if renorm else 0.0
    dmag = (np.abs(g64) * si).sum(1, keepdims=True) / total if renorm else 0.0
    want, mag = np.zeros((t, e)), np.zeros((t, e))
    np.put_along_axis(want, ids, 1.5 * (g64 - d) / total, 1)
    np.put_along_axis(mag, ids, 1.5 * (np.abs(g64) + dmag) / total, 1)
    want *= s * comp
    R.within("dlogits", out, want, 4 * R.route_precision(l)[:, None] * mag * s * comp + 2.0**-126)


@pytest.mark.parametrize("e,k", [(384, 8), (600, 20)])
def test_sigmoid_scores_below_the_normal_range(dev, e, k):
    """Scores of logits between -103 and -60 are fp32 numbers, the lowest in steps of 2^-149, and a large scale
    brings their weights and gradients back into sight."""
    _say("below the normal range", e, k)
    t, scale = 31, 1e22
    rng = np.random.default_rng(e)
    l = rng.uniform(-101, -88, (t, e)).astype(np.float32)
    router = dev.DeviceRouter(e, k, score="sigmoid", scale=scale)
    ids, w = router.forward(torch.from_numpy(l).cuda())
    want_ids, want, _ = R.route(l, k, score="sigmoid", scale=scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids) and want.max() > 1
    R.within("weights", w, want, 2 * R.route_precision(l)[:, None] * np.abs(want) + scale / 1e-20 * 2 * STEP)
    l = rng.uniform(-101, -60, (t, e)).astype(np.float32)
    prec = R.route_precision(l)[:, None]
    low = np.argsort(l, 1)[:, :k].copy()  # the smallest scores, most of them below 2^-126
    _, g = _slots(e, t, e, k)
    out = _gradient(dev, torch.from_numpy(l), low, g, score="sigmoid", scale=scale)
    want, _ = R.route_bwd(l, low, g, score="sigmoid", scale=scale)
    s = R.scores(l, "sigmoid")
    si, g64 = np.take_along_axis(s, low, 1), np.abs(g.astype(np.float64))
    total = si.sum(1, keepdims=True) + 1e-20
    mag = np.zeros((t, e))
    np.put_along_axis(mag, low, scale * (g64 + (g64 * si).sum(1, keepdims=True) / total) / total, 1)
    bound = mag * (4 * prec * s + 4 * STEP) + 2.0**-126
    assert (np.abs(want) > 4 * bound).any()  # values that a gradient of 0 would miss
    R.within("dlogits", out, want, bound)
