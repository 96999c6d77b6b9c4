"""GPU: norms before and after a block with its gate, scale and the residual stream, and their gradients, against a
plain 64-bit implementation.  Each case prints its name."""

import pytest

from tests import block_reference as R
from tests import step_reference as S

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[norm]", *a, flush=True)


def _make(seed, t, h, stream, branch=True, post=True, gate="channel", bias=True, weight=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    i = {"x": (n(t, h) * torch.exp(0.7 * n(h))).to(stream).cuda(), "branch": (n(t, h) * 0.5).to(BF16).cuda() if branch else None}
    i["token_gate"] = torch.rand(t, generator=g).cuda() if gate in ("token", "both") else None
    vec = lambda on, mean: (mean + 0.2 * n(h)).cuda() if on else None  # noqa: E731
    v = {"weight": vec(weight, 1.0), "bias": vec(bias, 0.0), "branch_weight": vec(post and weight, 1.0),
         "branch_bias": vec(post and bias, 0.0), "gate": vec(gate in ("channel", "both"), 0.5)}
    return i, v, n


def _forward(dev, i, v, kind, scale, post, **kw):
    norm = dev.DeviceNorm(i["x"].shape[1], kind, eps=1e-5, scale=scale, branch_norm=post, **v)
    h, y = norm.forward(i["x"], branch=i["branch"], token_gate=i["token_gate"], **kw)
    args = dict(kind=kind, eps=R.np.float32(1e-5).item(), scale=R.np.float32(scale).item(), branch_norm=post, **v)
    return norm, h, y, args


SIZES = [(1, 7168), (5, 1), (3, 7), (2, 8), (130, 64), (7, 512), (33, 513), (3, 520), (9, 2049), (700, 768), (5, 8192), (4, 8200),
         (3, 16384), (2, 16383)]


@pytest.mark.parametrize("t,h", SIZES)
@pytest.mark.parametrize("kind,stream,branch,post,gate,bias", [
    ("rms", BF16, True, True, "channel", False), ("rms", F32, True, False, "token", True), ("layer", BF16, True, True, "both", True),
    ("layer", F32, False, False, "none", True), ("rms", BF16, False, False, "none", False), ("rms", F32, True, True, "none", True)])
def test_forward_and_backward(dev, t, h, kind, stream, branch, post, gate, bias):
    _say(t, h, kind, stream, branch, post, gate, bias)
    i, v, n = _make(t + h, t, h, stream, branch, post, gate, bias)
    norm, hh, y, args = _forward(dev, i, v, kind, 0.75, post)
    want_h, dh, want_y, dy = S.norm_fwd(i["x"], i["branch"], i["token_gate"], **args)
    R.within("h", hh, want_h, dh + S.rounding(stream) * (want_h.abs() + dh))
    R.within("y", y, want_y, dy + R.UB * (want_y.abs() + dy))

    for with_h, with_y in ((True, True), (False, True), (True, False)):
        gh = n(t, h).to(stream).cuda() if with_h else None
        gy = n(t, h).to(BF16).cuda() if with_y else None
        old = {name: n(h).cuda() for name, x in v.items() if x is not None and (with_y or name not in ("weight", "bias"))}
        if branch:
            old.setdefault("gate", n(h).cuda())
        if not branch:
            old = {name: x for name, x in old.items() if name in ("weight", "bias")}
        grads = {name: x.clone() for name, x in old.items()}
        gtg = torch.empty(t, device="cuda") if i["token_gate"] is not None else None
        gx, gb = norm.backward(hh, norm.workspace(t), grads, branch=i["branch"], token_gate=i["token_gate"], grad_h=gh, grad_y=gy,
                               grad_token_gate=gtg, accumulate=True, grad_scale=0.5)
        want = S.norm_bwd(hh, i["branch"], i["token_gate"], gh, gy, **args)
        e, b = want["x"]
        R.within("grad_x", gx, e, b + S.rounding(stream) * (e.abs() + b))
        if branch:
            e, b = want["branch"]
            R.within("grad_branch", gb, e, b + R.UB * (e.abs() + b))
        else:
            assert gb is None
        if gtg is not None:
            e, b = want["token_gate"]
            R.within("grad_token_gate", gtg, e, b + R.U * e.abs())
        for name, x in grads.items():
            e, b = want[name]
            e = old[name].double().cpu() + 0.5 * e
            R.within(name, x, e, 0.5 * b + 2 * R.U * (e.abs() + old[name].double().cpu().abs()))


@pytest.mark.parametrize("t,h", [(600, 8193), (523, 16384)])
@pytest.mark.parametrize("kind,stream,bias", [("layer", F32, True), ("rms", BF16, False)])
def test_many_tokens_of_wide_rows(dev, t, h, kind, stream, bias):
    """Several rows a workgroup where not all of the vectors' gradients lie in registers."""
    _say("wide rows", t, h, kind, stream, bias)
    i, v, n = _make(t + h, t, h, stream, True, True, "both", bias)
    norm, hh, _, args = _forward(dev, i, v, kind, 0.75, True)
    gh, gy = n(t, h).to(stream).cuda(), n(t, h).to(BF16).cuda()
    grads, gtg = norm.grad_buffers(), torch.empty(t, device="cuda")
    gx, gb = norm.backward(hh, norm.workspace(t), grads, branch=i["branch"], token_gate=i["token_gate"], grad_h=gh, grad_y=gy, grad_token_gate=gtg)
    want = S.norm_bwd(hh, i["branch"], i["token_gate"], gh, gy, **args)
    for name, got, half in [("x", gx, S.rounding(stream)), ("branch", gb, R.UB), ("token_gate", gtg, R.U)] + [(k, x, 2 * R.U) for k, x in grads.items()]:
        e, b = want[name]
        R.within(name, got, e, b + half * (e.abs() + b))


def test_formula_against_differences(dev):
    """The reference's gradients, and with them the kernels', against central differences of its forward."""
    _say("differences")
    for kind in ("rms", "layer"):
        t, h = 3, 11
        i, v, n = _make(4, t, h, F32, True, True, "both", True)
        args = dict(kind=kind, eps=1e-3, scale=0.75, branch_norm=True, **v)
        hh = S.norm_fwd(i["x"], i["branch"], i["token_gate"], **args)[0]
        gh, gy = n(t, h).double(), n(t, h).double()
        want = S.norm_bwd(hh, i["branch"], i["token_gate"], gh, gy, **args)
        leaves = {"x": i["x"], "branch": i["branch"], "token_gate": i["token_gate"], **v}
        for name, value in leaves.items():
            base = value.double().cpu()
            for at in range(0, base.numel(), 3):
                f = []
                for step in (1e-5, -1e-5):
                    moved = base.clone()
                    moved.view(-1)[at] += step
                    a = {**leaves, name: moved}
                    hs, _, ys, _ = S.norm_fwd(a["x"], a["branch"], a["token_gate"], **{**args, **{k: a[k] for k in v}})
                    f.append(float((hs * gh).sum() + (ys * gy).sum()))
                got = float(want[name][0].reshape(-1)[at])
                assert abs((f[0] - f[1]) / 2e-5 - got) <= 1e-6 * (1 + abs(got)), (kind, name, at)


@pytest.mark.parametrize("h", [64, 7168, 100])
def test_in_place_and_missing_parts(dev, h):
    _say("in place", h)
    t = 37
    i, v, n = _make(8, t, h, F32, gate="both")
    norm, hh, y, _ = _forward(dev, i, v, "rms", 0.5, True)
    x = i["x"].clone()
    h2, y2 = norm.forward(x, branch=i["branch"], token_gate=i["token_gate"], h=x)
    assert h2 is x and torch.equal(x, hh) and torch.equal(y, y2)
    none, y3 = norm.forward(i["x"], branch=i["branch"], token_gate=i["token_gate"], need_h=False)
    assert none is None and torch.equal(y3, y)
    h4, none = norm.forward(i["x"], branch=i["branch"], token_gate=i["token_gate"], need_y=False)
    assert none is None and torch.equal(h4, hh)
    gh, gy, ws = n(t, h).cuda(), n(t, h).to(BF16).cuda(), norm.workspace(t)
    grads, some = norm.grad_buffers(), norm.grad_buffers()
    kw = dict(branch=i["branch"], token_gate=i["token_gate"], grad_y=gy)
    gx, gb = norm.backward(hh, ws, grads, grad_h=gh, **kw)
    g2 = gh.clone()
    gx2, gb2 = norm.backward(hh, ws, {"gate": some["gate"]}, grad_h=g2, grad_x=g2, **kw)
    assert gx2 is g2 and torch.equal(g2, gx) and torch.equal(gb2, gb) and torch.equal(some["gate"], grads["gate"])
    assert norm.backward(hh, ws, some, grad_h=gh, need_input=False, **kw) == (None, None)
    assert all(torch.equal(some[k], grads[k]) for k in grads)


@pytest.mark.parametrize("h", [513, 2049, 4099, 8191, 16383])
@pytest.mark.parametrize("stream", [BF16, F32])
def test_odd_rows_in_place(dev, h, stream):
    """Rows that are no whole chunks, of several waves, without a norm between the reads and the writes."""
    _say("odd rows in place", h, stream)
    t = 900
    i, v, n = _make(12, t, h, stream, post=False, gate="none", bias=False)
    norm = dev.DeviceNorm(h, **v)
    hh, y = norm.forward(i["x"], branch=i["branch"])
    gh = n(t, h).to(stream).cuda()
    gx, gb = norm.backward(hh, norm.workspace(t), {}, branch=i["branch"], grad_h=gh)
    for need_y in (False, True):
        x = i["x"].clone()
        _, y2 = norm.forward(x, branch=i["branch"], h=x, need_y=need_y)
        assert torch.equal(x, hh) and (y2 is None or torch.equal(y2, y))
    g2 = gh.clone()
    norm.backward(hh, norm.workspace(t), {}, branch=i["branch"], grad_h=g2, grad_x=g2)
    assert torch.equal(g2, gx)


@pytest.mark.parametrize("h", [96, 4096, 77])
def test_rows_alone_and_shorter_batches(dev, h):
    """A row's outputs do not depend on the batch; one workspace serves shorter batches; empty ones run the window rule."""
    _say("rows", h)
    t = 2100
    i, v, n = _make(9, t, h, BF16, gate="token")
    norm, hh, y, _ = _forward(dev, i, v, "layer", 1.5, True)
    ws = norm.workspace(t)
    gh, gy = n(t, h).to(BF16).cuda(), n(t, h).to(BF16).cuda()
    grads = norm.grad_buffers()
    gx, gb = norm.backward(hh, ws, grads, branch=i["branch"], token_gate=i["token_gate"], grad_h=gh, grad_y=gy)
    for s in (slice(0, 1), slice(3, 8), slice(1000, 1601)):
        kw = dict(branch=i["branch"][s], token_gate=i["token_gate"][s])
        if s.start * h * 2 % 16 or s.start * 4 % 4:
            continue
        h1, y1 = norm.forward(i["x"][s], **kw)
        assert torch.equal(h1, hh[s]) and torch.equal(y1, y[s])
        own, one = norm.grad_buffers(), norm.grad_buffers()
        a = norm.backward(hh[s], norm.workspace(s.stop - s.start), own, grad_h=gh[s], grad_y=gy[s], **kw)
        b = norm.backward(hh[s], ws, one, grad_h=gh[s], grad_y=gy[s], **kw)
        assert torch.equal(a[0], gx[s]) and torch.equal(a[1], gb[s])
        assert torch.equal(b[0], a[0]) and all(torch.equal(own[k], one[k]) for k in own)
    empty = i["x"][:0]
    h0, y0 = norm.forward(empty, branch=i["branch"][:0], token_gate=i["token_gate"][:0])
    assert h0.shape == y0.shape == (0, h)
    kept = {k: x.clone() for k, x in grads.items()}
    norm.backward(empty, ws, grads, branch=i["branch"][:0], grad_y=gy[:0], accumulate=True)
    assert all(torch.equal(grads[k], kept[k]) for k in grads)
    norm.backward(empty, ws, grads, branch=i["branch"][:0], grad_y=gy[:0])
    assert all(not x.any() for x in grads.values())


def test_values_that_are_not_finite_stay_in_their_row(dev):
    _say("not finite")
    t, h = 6, 264
    i, v, n = _make(10, t, h, F32, post=False, gate="none", bias=False)
    i["x"][1, 5], i["branch"][2, 7], i["x"][3, 0] = float("nan"), float("inf"), float("-inf")
    _, hh, y, _ = _forward(dev, i, v, "rms", 1.0, False)
    bad = torch.isnan(y.float()).any(1).cpu()
    assert bad.tolist() == [False, True, True, True, False, False]
    assert torch.isnan(hh[1, 5]) and torch.isinf(hh[2, 7]) and torch.isinf(hh[3, 0])
    # rows of zeros, and rows too small for fp32's squares: eps holds
    z = torch.zeros(2, h, device="cuda")
    z[1] = 1e-30
    _, y = dev.DeviceNorm(h, weight=v["weight"]).forward(z)
    assert not y.float().isnan().any() and not y[0].any()
