"""8-bit states of AdamW: codes are the nearest ones, ties to even, and bit for bit those of the kernel's formula in
elementary fp32 operations.  On the CPU: an encoder that truncates is told apart."""

import math

import pytest

from tests import step_reference as S
from tests.block_reference import U

torch = pytest.importorskip("torch")

F32, F64, BF16, E4M3 = torch.float32, torch.float64, torch.bfloat16, torch.float8_e4m3fn
BLOCK = 256


def _blocks(v):
    return torch.cat([v, v.new_zeros(-v.numel() % BLOCK)]).view(-1, BLOCK)


def _values(codes, scale):
    return (_blocks(codes.double()) * scale.double()[:, None]).view(-1)[: codes.numel()]


def off_the_nearest(codes, v, dv, root):
    """How far codes' values (a code of 1 is 1) lie from v times 448 / its block's largest, in bounds: half a step of
    E4M3 there, and what v is known to.  A neighbour of the nearest code passes where v lies within that of the middle."""
    pad, dpad = _blocks(v), _blocks(dv)
    amax = pad.abs().amax(1, keepdim=True)
    some = amax >= 2.0**-100
    by = torch.where(some, 448 / torch.where(some, amax, 1.0), 0.0)
    w = pad * by
    # the largest is known to its dv; scaling rounds four times
    dw = 1.1 * (dpad * by + w.abs() * (dpad.amax(1, keepdim=True) * by / 448 + 4 * U))
    if root:
        w = torch.where(w > 0, w.clamp(min=2.0**-9), w)
    off = (_blocks(codes.double()) - w).abs()
    # (a step that begins at a power of two: from below it is half as long)
    bound = S.e4m3_step(w) / 2 + dw
    return (off / bound.clamp(min=1e-300)).view(-1)[: v.numel()]


def truncated(v):
    """The planted mistake: codes toward 0."""
    w = _blocks(v)
    w = w / w.abs().amax(1, keepdim=True) * 448
    step = S.e4m3_step(w)
    return (torch.trunc(w / step) * step).view(-1)[: v.numel()]


def test_truncated_codes_are_told_apart():
    g = torch.Generator().manual_seed(1)
    v = torch.randn(1 << 14, generator=g, dtype=F64)
    dv = 4 * U * v.abs()
    q, scale, dq, _ = S.e4m3_blocks(v, dv, False)
    assert (off_the_nearest(q, v, dv, False) <= 1).all()
    bad = truncated(v)
    assert (off_the_nearest(bad, v, dv, False) > 1).double().mean() > 0.4
    assert ((bad - q).abs() <= dq).all()  # a bound of a whole step takes all of them
    assert abs(_drift(q, v)) < 0.02 and _drift(bad, v) < -0.3


def _drift(codes, v):
    """The mean of how far codes lie from their values, away from 0, in steps."""
    w = _blocks(v)
    w = (w / w.abs().amax(1, keepdim=True) * 448).view(-1)[: v.numel()]
    return float(((codes.double() - w) * w.sign() / S.e4m3_step(w)).mean())


# ---------------------------------------------------------------- GPU


def _f(x):
    return torch.tensor(x, dtype=F64).to(F32)


# Roots and quotients in 64 bits, then rounded: exact to half a step, since 53 >= 2 * 24 + 2 (torch's own roots on the CPU are
# off by a step in one of six).
def _root(v):
    return v.double().sqrt().float()


def _over(a, b):
    return (a.double() / b.double()).float()


def encode(v, root):
    """Codes and scales as the kernel makes them, in fp32."""
    b = _blocks(v)
    amax = b.abs().amax(1)
    some = amax >= 2.0**-100
    inv = torch.where(some, _f(448.0) * _over(_f(1.0), amax), 0.0)
    w = b * inv[:, None]
    if root:
        w = torch.where((b > 0) & some[:, None], w.clamp(min=2.0**-9), w)
    return w.clamp(-448, 448).to(E4M3).view(-1)[: v.numel()], torch.where(some, amax * _f(1 / 448), 0.0)


def step32(p, g, m, v, m_scale, v_scale, t, lr, betas, eps, decay, grad_scale):
    """One step in elementary fp32 operations, each rounded, in the formula's order: (p, (m, scales), (v, scales))."""
    rows = lambda s: s.repeat_interleave(BLOCK)[: p.numel()]  # noqa: E731
    b1, b2 = betas
    g = g.float() * _f(grad_scale)
    m = m.float() * rows(m_scale)
    v = v.float() * rows(v_scale)
    v = v * v
    m = _f(b1) * m + _f(1 - b1) * g
    v = _f(b2) * v + _f(1 - b2) * (g * g)
    root = _root(v)
    c1, c2 = 1 - b1**t, 1 - b2**t
    p = p.float() * _f(1 - lr * decay) - _over(_f(lr / c1) * m, root * _f(1 / math.sqrt(c2)) + _f(eps))
    return p, encode(m, False), encode(root, True)


def _same(name, got, want):
    got, want = got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)
    assert torch.equal(got, want), f"{name}: {int((got != want).sum())} bytes of {got.numel()} differ"


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 255, 257, 4096, 70001, 300000])
@pytest.mark.parametrize("dtype,master", [(F32, False), (BF16, False), (BF16, True)])
@pytest.mark.parametrize("grad", [F32, BF16])
def test_codes_of_the_formula(dev, n, dtype, master, grad):
    """Three steps (beta1 = 0.5 and 0.75: powers that no way of multiplying rounds), bit for bit; every code the nearest; no drift."""
    print("[adamw codes]", n, dtype, master, grad, flush=True)
    g = torch.Generator().manual_seed(n)
    p = (torch.randn(n, generator=g) * 0.05).to(dtype)
    hyper = dict(lr=2e-3, betas=(0.5, 0.75), eps=1e-7, weight_decay=0.1)
    opt = dev.DeviceAdamW({"w": p.cuda()}, states="e4m3", master=master, **hyper)
    s = opt.state["w"]
    for t in range(1, 4):
        grads = (torch.randn(n, generator=g) * 4.0 ** torch.randint(-6, 3, (n,), generator=g)).to(grad)
        old = {k: x.cpu() for k, x in s.items()}
        before = old["master"] if master else opt.params["w"].cpu()
        opt.step({"w": grads.cuda()}, grad_scale=0.5)
        want, (m, m_scale), (v, v_scale) = step32(before, grads, old["m"], old["v"], old["m_scale"], old["v_scale"], t, hyper["lr"], hyper["betas"],
                                                  hyper["eps"], hyper["weight_decay"], 0.5)
        _same("m", s["m"], m), _same("m_scale", s["m_scale"], m_scale)
        _same("v", s["v"], v), _same("v_scale", s["v_scale"], v_scale)
        _same("param", opt.params["w"], want.to(dtype))
        if master:
            _same("master", s["master"], want)
        # against 64 bits: the moments to a few roundings
        m0, v0 = _values(old["m"], old["m_scale"]), _values(old["v"], old["v_scale"]) ** 2
        gd = grads.double() * 0.5
        m64, v64 = 0.5 * m0 + 0.5 * gd, 0.75 * v0 + 0.25 * gd * gd
        dm = 4 * U * ((0.5 * m0).abs() + (0.5 * gd).abs())
        for key, value, dvalue, root in (("m", m64, dm, False), ("v", v64.sqrt(), 6 * U * v64.sqrt(), True)):
            worst = off_the_nearest(s[key].cpu(), value, dvalue, root)
            assert float(worst.max()) <= 1, key
        # The mean of a rounding to the nearest, in steps: 0 to 1 / sqrt(12 n) where values are spread evenly over a step.  At a power of two a code
        # takes half a step from above (a mean of -1/4) and a quarter from below (1/4 of the shorter step): -1/16 of a step among 8, 0.008.
        # Values whose density falls as 1 / w lie unevenly by a step / w of 1/8 at most, 1/12 of which is 0.010.  Truncation: -0.5.
        if n >= 70000:
            large = m64.abs() > 2.0**-5 * _blocks(m64).abs().amax(1).repeat_interleave(BLOCK)[:n]
            w = m64 * (448 / _blocks(m64).abs().amax(1)).repeat_interleave(BLOCK)[:n]
            drift = ((s["m"].cpu().double() - w) * w.sign() / S.e4m3_step(w))[large]
            assert abs(float(drift.mean())) <= 0.02 + 6 / math.sqrt(12 * drift.numel())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0, -30, 17, -108, -109])
def test_ties_subnormals_and_the_least_root(dev, scale):
    """beta1 = beta2 = 0: m is the gradient and sqrt(v) its magnitude.  All middles of E4M3's codes and a hair to both sides of them, with the largest
    448 in their block: nearest, ties to even; roots that would be 0 keep the least code; blocks below 2^-100 are zeros."""
    print("[adamw codes] ties", scale, flush=True)
    codes = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double()  # 0 to 448
    middles = (codes[1:] + codes[:-1]) / 2
    # (a middle has 5 bits, its square 10: both exact in fp32, as is a hair of 2^-10 of it, 15 bits)
    w = torch.cat([codes, middles, middles * (1 - 2.0**-10), middles * (1 + 2.0**-10), torch.tensor([2.0**-12, 2.0**-20])])
    w = w[w <= 448]
    parts = []
    for c in w.split(254):
        parts += [c, torch.zeros(254 - c.numel(), dtype=F64), torch.tensor([448.0, -448.0], dtype=F64)]
    w = torch.cat(parts)
    w[1::3] *= -1
    g = (w * 2.0**scale).float()
    assert torch.equal(g.double(), w * 2.0**scale)
    opt = dev.DeviceAdamW({"w": torch.zeros(w.numel(), device="cuda")}, betas=(0.0, 0.0), states="e4m3", weight_decay=0.0)
    opt.step({"w": g.cuda()})
    s = {k: x.cpu() for k, x in opt.state["w"].items()}
    if scale == -109:  # 448 times that is 2^-100.2 (and its square no fp32 number)
        assert not s["m"].float().any() and not s["m_scale"].any() and not s["v_scale"].any()
        return
    assert torch.equal(s["m_scale"].double(), torch.full_like(s["m_scale"], 2.0**scale, dtype=F64))
    _same("m", s["m"], w.float().to(E4M3))
    root = w.abs()
    want = torch.where(root > 0, root.clamp(min=2.0**-9), 0.0)
    if scale == 0:  # (elsewhere the squares of the least leave fp32)
        _same("v", s["v"], want.float().to(E4M3))
        assert ((s["v"].float() > 0) == (root > 0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 2.0**65])
def test_a_moment_that_is_not_finite_stays_in_its_block(dev, value):
    """Without the check for finite gradients: every other block is as if nothing had been."""
    print("[adamw codes] not finite", value, flush=True)
    g = torch.Generator().manual_seed(3)
    p, grads = torch.randn(3000, generator=g).cuda(), [torch.randn(3000, generator=g).cuda() for _ in range(2)]
    runs = []
    for bad in (False, True):
        opt = dev.DeviceAdamW({"w": p.clone()}, states="e4m3")
        for i, x in enumerate(grads):
            x = x.clone()
            if bad and i == 0:
                x[700] = value
            opt.step({"w": x})
        runs.append((opt.params["w"], opt.state["w"]))
    (a, s), (b, q) = runs
    other = torch.ones(3000, dtype=torch.bool, device="cuda")
    other[512:768] = False
    assert torch.equal(a[other], b[other]) and torch.isfinite(b[other]).all()
    v = q["v"][700].float() * q["v_scale"][2]
    assert not torch.isfinite(v)
    for k in ("m", "v"):
        assert torch.equal(s[k].view(torch.uint8)[other], q[k].view(torch.uint8)[other])
