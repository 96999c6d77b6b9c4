"""GPU: the norms' gradients where a workgroup or a team of waves takes several rows, one of them ahead of the other, against the
plain 64-bit implementation (every width that a rule of the kernels names, and both sides of it).  Each case prints its name."""

import pytest

from tests import block_reference as R
from tests import step_reference as S
from tests.test_norm import BF16, F32, _forward, _make

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


# tokens: more than 256 workgroups of one row (above 4096 columns) or of all teams (16 / waves of them); a last round in which some teams
# have no row
@pytest.mark.parametrize("t,h", [(257, 4097), (600, 4104), (523, 7168), (771, 8192), (300, 8191),
                                 (1100, 4096), (1541, 2049), (2050, 2048), (2700, 1025), (4099, 520), (4200, 512), (9001, 64), (8300, 7), (4097, 1)])
@pytest.mark.parametrize("kind,stream,branch,post,gate,bias", [
    ("layer", F32, True, True, "both", True), ("rms", BF16, True, True, "channel", False), ("rms", BF16, True, False, "token", True),
    ("layer", BF16, False, False, "none", True)])
def test_several_rounds(dev, t, h, kind, stream, branch, post, gate, bias):
    print("[norm rounds]", t, h, kind, stream, branch, post, gate, bias, flush=True)
    i, v, n = _make(t + h, t, h, stream, branch, post, gate, bias)
    norm, hh, _, args = _forward(dev, i, v, kind, 0.75, post)
    if not branch:
        hh = i["x"]
    gh, gy = n(t, h).to(stream).cuda(), n(t, h).to(BF16).cuda()
    grads = norm.grad_buffers()
    gtg = torch.empty(t, device="cuda") if i["token_gate"] is not None else None
    ws = norm.workspace(t)
    kw = dict(branch=i["branch"], token_gate=i["token_gate"], grad_h=gh, grad_y=gy, grad_token_gate=gtg)
    gx, gb = norm.backward(hh, ws, grads, **kw)
    want = S.norm_bwd(hh, i["branch"], i["token_gate"], gh, gy, **args)
    got = [("x", gx, S.rounding(stream))] + [(k, x, 2 * R.U) for k, x in grads.items()]
    if branch:
        got.append(("branch", gb, R.UB))
    if gtg is not None:
        got.append(("token_gate", gtg, R.U))
    for name, x, half in got:
        e, b = want[name]
        R.within(name, x, e, b + half * (e.abs() + b))
    again = norm.grad_buffers(fill=float("nan"))
    ws.fill_(0x7F)
    norm.backward(hh, ws, again, **kw)
    assert all(torch.equal(again[k], grads[k]) for k in grads)
