"""GPU: routing of tokens to experts and its gradient, against a plain 64-bit
implementation.  The choice must be equal; weights and gradients lie within
the bounds derived in block_reference.  Each case prints its name first."""

import numpy as np
import pytest

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
    print("[router]", *a, flush=True)


def _logits(seed, t, e, std=1.5, bf16=False):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(t, e, generator=g) * std
    return l.to(torch.bfloat16) if bf16 else l


def _bias(seed, e, std=0.1):
    return torch.randn(e, generator=torch.Generator().manual_seed(seed + 999)) * std


def _check(dev, logits, top_k, bias=None, mask=None, load=True, **cfg):
    router = dev.DeviceRouter(logits.shape[1], top_k, bias=None if bias is None else bias.cuda(), **cfg)
    t, e = logits.shape
    got_load = torch.full((e,), 7, dtype=torch.int32, device="cuda") if load else None
    ids = torch.full((t, top_k), -5, dtype=torch.int64, device="cuda")
    w = torch.full((t, top_k), 5.0, device="cuda")
    router.forward(logits.cuda(), token_mask=None if mask is None else mask.cuda(), expert_ids=ids, route_weights=w,
                   load=got_load)
    torch.cuda.synchronize()
    want_ids, want_w, want_load = R.route(logits.float().numpy(), top_k, bias=None if bias is None else bias.numpy(),
                                          mask=None if mask is None else mask.numpy(), **cfg)
    assert np.array_equal(ids.cpu().numpy(), want_ids), "another choice"
    bound = 2 * R.route_precision(logits.float().numpy())[:, None] * np.abs(want_w) + 2.0**-140
    R.within("weights", w, want_w, np.where(np.isnan(bound), 0, bound))
    if load:
        assert np.array_equal(got_load.cpu().numpy(), want_load)
    return router, ids, w


SHAPES = [
    (1, 1, 1), (3, 2, 1), (5, 7, 7), (33, 16, 4), (17, 60, 4), (9, 64, 6), (130, 96, 3), (64, 128, 8), (31, 160, 6),
    (257, 256, 8), (300, 384, 8), (65, 384, 16), (12, 384, 17), (21, 511, 5), (19, 512, 10), (11, 513, 9), (6, 1000, 64),
    (3, 8192, 8), (2, 8192, 300),
]


@pytest.mark.parametrize("t,e,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_choice_and_weights(dev, t, e, k, score, bf16, biased):
    _say("choice", t, e, k, score, bf16, biased)
    _check(dev, _logits(t + e, t, e, bf16=bf16), k, bias=_bias(e, e) if biased else None, score=score,
           renormalize=bf16 != biased, scale=2.5 if biased else 1.0)


@pytest.mark.parametrize("e,groups,top_groups,group_top,k", [
    (384, 8, 4, 2, 8), (384, 8, 4, 1, 8), (256, 8, 4, 2, 8), (256, 8, 1, 2, 8), (160, 8, 3, 1, 6), (64, 4, 2, 2, 6),
    (60, 4, 2, 2, 6), (24, 8, 3, 2, 8), (16, 16, 5, 1, 5), (128, 64, 40, 2, 12), (8, 2, 2, 2, 3), (1024, 16, 4, 2, 10),
    (512, 2, 1, 2, 16), (32, 2, 1, 2, 16), (104, 8, 5, 2, 12), (96, 3, 2, 2, 7), (85, 5, 2, 1, 11), (117, 9, 4, 2, 9),
    (320, 10, 3, 2, 8), (480, 15, 7, 2, 16), (26, 13, 6, 2, 4), (512, 16, 4, 2, 8), (136, 17, 4, 2, 8), (528, 16, 4, 2, 8),
])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(dev, e, groups, top_groups, group_top, k, score, biased):
    _say("groups", e, groups, top_groups, group_top, k, score, biased)
    _check(dev, _logits(e + k, 203, e, bf16=group_top == 1), k, bias=_bias(e, e) if biased else None, score=score,
           num_groups=groups, top_groups=top_groups, group_top=group_top, scale=2.5)


@pytest.mark.parametrize("e,groups,top_groups", [(384, 1, 1), (384, 8, 4), (60, 1, 1), (600, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_neighbours(dev, e, groups, top_groups, score):
    """Equal scores go to the lower index; scores that fp32 cannot tell apart are told apart."""
    _say("ties", e, groups, score)
    rng = np.random.default_rng(e + groups)
    cfg = dict(score=score, num_groups=groups, top_groups=top_groups, group_top=1 if groups == 1 else 2)
    ties = torch.from_numpy(rng.integers(-2, 3, (120, e)).astype(np.float32))
    ties[0] = 0.25  # all equal
    ties[1] = torch.finfo(torch.float32).min
    ties[2] = torch.finfo(torch.bfloat16).min
    ties[2, 1::3] = torch.finfo(torch.float32).min
    _check(dev, ties, 8, **cfg)
    _check(dev, ties.to(torch.bfloat16), 8, **cfg)
    _check(dev, ties, 8, bias=torch.zeros(e), **cfg)
    _check(dev, ties, 8, bias=torch.from_numpy(rng.integers(-1, 2, e).astype(np.float32)), **cfg)
    # logits a step of fp32 apart
    base = rng.standard_normal((200, 1)).astype(np.float32)
    near = torch.from_numpy((base + rng.integers(-4, 5, (200, e)).astype(np.float32) * np.abs(base) * 2.0**-23))
    _check(dev, near, 8, **cfg)
    # c = s + b close to a constant: the bias takes back what the score gives, up to its own rounding
    l = rng.standard_normal(e).astype(np.float32)
    b = torch.from_numpy((0.5 - R.scores(l[None], score)[0]).astype(np.float32))
    rows = torch.from_numpy(np.repeat(l[None], 64, 0))
    rows[1:] += torch.from_numpy(rng.integers(-2, 3, (63, e)).astype(np.float32)) * 2.0**-22
    _check(dev, rows, 8, bias=b, **cfg)


@pytest.mark.parametrize("e,k", [(384, 8), (40, 6), (700, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 2])
def test_masks_infinities_and_nans(dev, e, k, score, groups):
    _say("masks", e, k, score, groups)
    l = _logits(e, 40, e)
    l[0] = -np.inf  # nobody left
    l[1] = -np.inf
    l[1, 3] = 0.5  # one left
    l[2, ::2] = -np.inf
    l[3, 5] = np.nan
    l[4, e - 1] = np.inf
    l[5] = np.nan
    l[6, : e - k + 2] = -np.inf  # fewer than k left
    l[7] *= 60  # scores from 1 down to 0
    l[8, 0] = 3e38
    l[9] = -200.0  # every sigmoid underflows
    l[10] = 200.0
    l[11, 1] = -np.inf
    mask = torch.ones(40, dtype=torch.bool)
    mask[[5, 20, 39]] = False
    cfg = dict(score=score, num_groups=groups, top_groups=1, group_top=2 if groups == 2 else 1)
    for bias in (None, _bias(1, e)):
        for m in (None, mask, mask.to(torch.uint8) * 3):
            _check(dev, l, k, bias=bias, mask=m, **cfg)
    out = _bias(2, e)
    out[: e // 4] = -np.inf  # experts out of service
    _check(dev, l, k, bias=out, mask=mask, **cfg)
    out[:] = -np.inf
    _check(dev, l, k, bias=out, **cfg)
    for v in (np.nan, np.inf):
        b = _bias(3, e)
        b[e // 2] = v
        _check(dev, l, k, bias=b, mask=mask, **cfg)


@pytest.mark.parametrize("e,k", [(384, 8), (600, 20)])
def test_scores_that_vanish_under_a_large_scale(dev, e, k):
    """Every s is 0 in fp32: the weights are 0 however large scale / 1e-20 is."""
    _say("large scale", e, k)
    _check(dev, _logits(9, 37, e) - 300, k, score="sigmoid", scale=1e25)


def test_no_tokens_and_load_window(dev):
    _say("load")
    router = dev.DeviceRouter(48, 4, score="sigmoid")
    load = torch.full((48,), 9, dtype=torch.int32, device="cuda")
    ids, w = router.forward(torch.empty(0, 48, device="cuda"), load=load, accumulate=True)
    assert ids.shape == (0, 4) and w.shape == (0, 4) and int(load.sum()) == 9 * 48
    router.forward(torch.empty(0, 48, device="cuda"), load=load)
    assert int(load.abs().sum()) == 0
    dl = router.backward(torch.empty(0, 48, device="cuda"), ids, w)
    assert dl.shape == (0, 48)
    for t in (100, 9000):
        l = _logits(t, t, 48).cuda()
        load.fill_(5)
        ids, _ = router.forward(l, load=load, accumulate=True)
        want = torch.bincount(ids.flatten(), minlength=48) + 5
        assert torch.equal(load.long(), want)
        router.forward(l, load=load)
        assert torch.equal(load.long(), want - 5)


@pytest.mark.parametrize("e", [1, 5, 384, 8192])
def test_bias_update(dev, e):
    _say("bias", e)
    rng = np.random.default_rng(e)
    load = rng.integers(0, 9, e).astype(np.int32)
    load[: e // 3] = int(load.mean())
    if e == 5:
        load[:] = 2**31 - 1
    b = _bias(4, e)
    router = dev.DeviceRouter(e, 1, bias=b.cuda())
    router.update_bias(torch.from_numpy(load).cuda(), 0.001)
    step = np.sign(int(load.astype(np.int64).sum()) - load.astype(np.int64) * e).astype(np.float32)
    assert np.array_equal(router.bias.cpu().numpy(), b.numpy() + step * np.float32(0.001))


# ---------------------------------------------------------------- gradient


def _check_bwd(dev, logits, ids, g, **cfg):
    router = dev.DeviceRouter(logits.shape[1], ids.shape[1], **cfg)
    out = torch.full(logits.shape, 3.0, dtype=logits.dtype, device="cuda")
    router.backward(logits.cuda(), ids.cuda(), g.cuda(), grad_logits=out)
    want, bound = R.route_bwd(logits.float().numpy(), ids.numpy(), g.numpy(), **cfg)
    # 2^-126: results below fp32's normal range may lose bits
    R.within("dlogits", out, want, bound + R.rounding(logits.dtype) * np.abs(want) + 2.0**-126)
    return out


@pytest.mark.parametrize("t,e,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient(dev, t, e, k, score, renorm):
    _say("gradient", t, e, k, score, renorm)
    for bf16 in (False, True):
        l = _logits(t + 2 * e, t, e, bf16=bf16)
        rng = np.random.default_rng(t + e)
        ids = torch.from_numpy(np.stack([rng.permutation(e)[:k] for _ in range(t)]))
        g = torch.from_numpy(rng.standard_normal((t, k)).astype(np.float32))
        _check_bwd(dev, l, ids, g, score=score, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("e,k", [(384, 8), (50, 6), (900, 5), (384, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_unusual_slots(dev, e, k, score, renorm):
    """Dropped and repeated ids, ids far out of range, undefined rows, rows of -inf."""
    _say("gradient slots", e, k, score, renorm)
    rng = np.random.default_rng(e)
    l = _logits(e, 24, e)
    ids = torch.from_numpy(np.stack([rng.permutation(e)[:k] for _ in range(24)]))
    g = torch.from_numpy(rng.standard_normal((24, k)).astype(np.float32))
    ids[0] = -1
    ids[1, 1:] = -1
    ids[2, 0] = e
    ids[3, 0] = 2**40
    ids[3, 1] = -(2**62)
    ids[4] = ids[4, 0]  # the same expert in every slot
    ids[5, 1] = ids[5, 0]
    l[6, 3] = np.nan
    l[7] = np.nan
    ids[7] = -1
    g[7] = np.nan
    l[8, 2] = np.inf
    l[9, ::2] = -np.inf
    l[10] *= 40
    ids[11, 2] = -1
    g[11, 2] = np.nan  # belongs to nobody
    g[12] = 0
    for bf16 in (False, True):
        _check_bwd(dev, l.to(torch.bfloat16) if bf16 else l, ids, g, score=score, renormalize=renorm, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(dev, score, renorm):
    """Central differences of the forward's own weights at a fixed choice, in fp32: step h gives an error of
    about h^2 of the third derivative (below 1, scores of one unit of logit) and 2^-23 / h of rounding."""
    _say("differences", score, renorm)
    e, k, t, h = 24, 4, 5, 2.0**-7
    cfg = dict(score=score, renormalize=renorm, scale=1.5)
    router = dev.DeviceRouter(e, k, **cfg)
    l = _logits(77, t, e)
    l = torch.round(l * 4) / 4 + torch.arange(e) * 0.0625  # distinct and more than 2 h apart where chosen
    ids, _ = router.forward(l.cuda())
    g = torch.randn(t, k, generator=torch.Generator().manual_seed(1))
    dl = router.backward(l.cuda(), ids, g.cuda()).cpu()
    for j in range(e):
        side = []
        for sign in (1, -1):
            moved = l.clone()
            moved[:, j] += sign * h
            i2, w2 = router.forward(moved.cuda())
            side.append((i2.cpu(), w2.cpu()))
        same = (torch.sort(side[0][0], 1).values == torch.sort(ids.cpu(), 1).values).all(1) & \
               (torch.sort(side[1][0], 1).values == torch.sort(ids.cpu(), 1).values).all(1)
        val = []
        for i2, w2 in side:
            full = torch.zeros(t, e).scatter_(1, i2, w2)
            val.append((full.gather(1, ids.cpu()) * g).sum(1))
        num = (val[0] - val[1]) / (2 * h)
        scale = 1.5 * g.abs().sum(1)
        assert (torch.where(same, (num - dl[:, j]).abs(), 0.0) <= scale * (h * h + 2.0**-21 / h)).all()
        assert same.float().mean() > 0.5
