"""Gradients of dense products from a dz that bf16 does not hold (an fp32
grad_output, or one times an activation's slope), which enters the products as
bf16 numbers that sum to it.  GPU tests against 64-bit products, and CPU tests
that the bounds tell fewer planes from enough.  Each case prints its name first.

dz = p0 + p1 + p2: p0 and p1 are cut off after their 8 significant bits, so p2
holds the rest of the 24 exactly (for |dz| above 2^-100): d_weight takes no
error from the planes.  grad_input takes p0 and the rest rounded to bf16: the
rest is at most a step of p0, 2^-7 |dz|, and below that step in the binades
under it, so half a step of the rest is at most 2^-16 |dz|.
"""

import math

import pytest

from tests import block_reference as R

torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
REST = 2.0**-16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[planes]", *a, flush=True)


def _rand(seed, *shape, std=1.0, dtype=BF16, where="cuda"):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(where)


def _dz(dy, z, act):
    """dz in 64 bits and the error of an fp32 evaluation of it (block_reference's)."""
    d = dy.double().cpu()
    if act == "none":
        return d, torch.zeros_like(d)
    return d * R.act_grad(z.double().cpu(), act), 32 * R.U * d.abs() * 1.2


FORMS = [("none", F32), ("silu", BF16), ("gelu", F32)]


# ---------------------------------------------------------------- grad_input


@gpu
@pytest.mark.parametrize("t,k,n", [(5, 8, 8), (33, 64, 40), (200, 264, 136), (64, 512, 72), (3471, 3656, 75)])
@pytest.mark.parametrize("act,dtype", FORMS)
def test_grad_input_takes_more_than_bf16_of_dz(dev, t, k, n, act, dtype):
    """Each column of W holds a single 1, and the residual takes dz's bf16 value away: what is left is what
    bf16 does not hold of dz."""
    _say("what is left", t, k, n, act, dtype)
    w = torch.zeros(n, k, dtype=BF16)
    w[torch.arange(k) % n, torch.arange(k)] = 1
    dy = _rand(1, t, n, dtype=dtype)
    z = _rand(2, t, n) if act != "none" else None
    dz, err = _dz(dy, z, act)
    picked, err = dz[:, torch.arange(k) % n], err[:, torch.arange(k) % n]
    res = (-picked).float().to(BF16)
    lin = dev.DeviceLinear(w.cuda(), None, act)
    dx = lin.backward(_rand(3, t, k), dy, lin.backward_workspace(t), {}, preact=z, grad_residual=res.cuda())
    want = picked + res.double()
    # two terms and the residual are added in fp32
    R.within("dx", dx, want, err + (REST + 3 * R.U) * picked.abs() + R.UB * want.abs())


@gpu
@pytest.mark.parametrize("t,k,n", [(1, 8, 1), (15, 136, 33), (31, 1024, 384), (65, 264, 130), (127, 96, 250),
                                   (300, 512, 384), (513, 1000, 257), (1025, 128, 520), (3471, 3656, 75),
                                   (75, 3656, 3471), (130, 3656, 3472)])
@pytest.mark.parametrize("act,dtype", FORMS)
def test_gradients_of_shapes(dev, t, k, n, act, dtype):
    """Both gradients with the planes' own errors, at every tile and split; alone they are the same bits."""
    _say("shapes", t, k, n, act, dtype)
    x, w, dy = _rand(1, t, k), _rand(2, n, k, std=n**-0.5), _rand(3, t, n, dtype=dtype)
    z = _rand(4, t, n) if act != "none" else None
    lin = dev.DeviceLinear(w, None, act)
    ws = lin.backward_workspace(t)
    ws.fill_(0xFF)
    grads = lin.grad_buffers(fill=0.5)
    dx = lin.backward(x, dy, ws, grads, preact=z)
    ws.fill_(0xFF)
    assert torch.equal(lin.backward(x, dy, ws, {}, preact=z), dx)
    alone = lin.grad_buffers(fill=0.5)
    ws.fill_(0xFF)
    lin.backward(x, dy, ws, alone, preact=z, need_input=False)
    assert torch.equal(alone["weight"], grads["weight"])
    dz, err = _dz(dy, z, act)
    xd, wd = x.double().cpu(), w.double().cpu()
    want, mag = dz @ wd, dz.abs() @ wd.abs()
    R.within("dx", dx, want, err @ wd.abs() + (REST + 8 * math.sqrt(2 * n) * R.U) * mag + R.UB * want.abs())
    want, mag = dz.t() @ xd, dz.abs().t() @ xd.abs()
    R.within("dw", grads["weight"], want, err.t() @ xd.abs() + (8 * math.sqrt(3 * t) + 1) * R.U * mag)


# ---------------------------------------------------------------- d_weight


def _few_planes(dy, planes, nearest):
    """dy from its first bf16 planes, on the CPU."""
    rest, total = dy.clone(), torch.zeros_like(dy, dtype=torch.float64)
    for _ in range(planes):
        h = rest.to(BF16).float() if nearest else (rest.view(torch.int32) & ~0xFFFF).view(F32)
        total += h.double()
        rest = rest - h
    return total


def _one_token(t, n, k):
    """A gradient with all 24 bits in use and inputs that are powers of two: one product (or, with two tokens
    of the same sign, two) whose planes' products are exact, so three roundings of sums are all there is."""
    dy = _rand(5, t, n, dtype=F32, where="cpu").abs() + 0.25
    dy = (dy.view(torch.int32) | 1).view(F32)
    x = torch.exp2(torch.randint(-6, 7, (t, k), generator=torch.Generator().manual_seed(6)).float()).to(BF16)
    want = dy.double().t() @ x.double()
    return dy, x, want, 4 * t * R.U * want


@pytest.mark.parametrize("t", [1, 2])
@pytest.mark.parametrize("nearest", [False, True])
def test_two_planes_are_told_from_three(t, nearest):
    dy, x, want, bound = _one_token(t, 40, 64)
    off = (_few_planes(dy, 2, nearest).t() @ x.double() - want).abs()
    assert (off > bound).float().mean() > 0.2
    assert ((_few_planes(dy, 3, nearest).t() @ x.double() - want).abs() <= bound).all()


@gpu
@pytest.mark.parametrize("t,k,n", [(1, 64, 40), (2, 64, 40), (1, 3656, 3471), (2, 264, 130)])
def test_weight_gradient_holds_all_of_dz(dev, t, k, n):
    _say("24 bits", t, k, n)
    dy, x, want, bound = _one_token(t, n, k)
    lin = dev.DeviceLinear(_rand(1, n, k))
    grads = lin.grad_buffers()
    lin.backward(x.cuda(), dy.cuda(), lin.backward_workspace(t), grads, need_input=False)
    R.within("dw", grads["weight"], want, bound)


# ---------------------------------------------------------------- infinities


@gpu
@pytest.mark.parametrize("t,k,n", [(9, 64, 40), (200, 264, 130), (130, 3656, 3472)])
@pytest.mark.parametrize("act,dtype", FORMS + [("none", BF16)])
def test_infinite_operands(dev, t, k, n, act, dtype):
    """A nonzero dz times an infinite input or weight is infinite, whether bf16 holds the dz or not; zeros, NaNs
    and infinities of both signs give what the products in 64 bits give."""
    _say("infinite operands", t, k, n, act, dtype)
    inf = float("inf")
    x, w, dy = _rand(1, t, k), _rand(2, n, k), _rand(3, t, n, dtype=dtype)
    x[3, 5], x[4, 7], x[5, 7] = inf, -inf, inf
    w[11, 9], w[12, 20] = inf, -inf
    dy[:, 1] = 1.0  # held by bf16
    dy[:, 2] = -2.5
    dy[:, 3] = 2.0**-99
    dy[3, 4] = 0.0
    dy[5, 6] = -inf
    if dtype is F32:
        dy[:, 14] = 1 + 2.0**-8  # held by two planes
        dy[:, 15] = 1e30
    z = _rand(4, t, n) if act != "none" else None
    lin = dev.DeviceLinear(w, None, act)
    grads = lin.grad_buffers()
    dx = lin.backward(x, dy, lin.backward_workspace(t), grads, preact=z)
    dz, _ = _dz(dy, z, act)
    xd, wd = x.double().cpu(), w.double().cpu()

    def check(tag, actual, want):
        """The same NaNs, the same infinities, and no others."""
        a = actual.double().cpu()
        assert torch.equal(torch.isnan(a), torch.isnan(want)), f"{tag}: NaNs at other places"
        at = torch.isinf(want)
        assert torch.equal(a[at], want[at]), f"{tag}: infinities"
        assert torch.isfinite(a[torch.isfinite(want)]).all(), f"{tag}: infinities at other places"

    check("dw", grads["weight"], dz.t() @ xd)
    check("dx", dx, dz @ wd)
