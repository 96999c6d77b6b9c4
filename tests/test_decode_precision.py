"""GPU: what lies between gate and up and down of the experts for a few tokens keeps fp32's digits: outputs that are
the difference of two nearly equal values.  Each case prints its name."""

import pytest

from int4_quantized_moe_amd import workloads as W
from tests import block_reference as R
from tests import step_reference as S

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
# nibbles: the largest number, its negative, zero, and what a second input of 1/32 is multiplied by
CODES = {"rawint4": (15, 1, 8, 9), "mxfp4": (7, 15, 0, 1)}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _pack(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8).contiguous()


# one kernel of gate and up and the other (up to 2048 wide and slots x intermediate from 12288 on), more than two slots an expert
# (a wave of down a slot), down split and not, contractions that end inside a chunk
@pytest.mark.parametrize("t,e,k,h,i", [(1, 4, 1, 64, 64), (3, 4, 2, 4096, 96), (8, 16, 2, 96, 1056), (33, 4, 2, 64, 224), (2, 3, 3, 64, 4128),
                                       (64, 8, 1, 64, 32)])
@pytest.mark.parametrize("fmt", ["rawint4", "mxfp4"])
@pytest.mark.parametrize("r", [0, 8])
def test_differences_keep_their_digits(dev, t, e, k, h, i, fmt, r):
    """Columns of h in pairs: up of one is w x, of the other w x + v x / 32, gate the same.  A row of down has a weight and its negative
    for a pair, so that the output is 1/100 to 1/400 of what is subtracted, and would lose its digits with an h of 11 bits."""
    print("[decode precision]", t, e, k, h, i, fmt, r, flush=True)
    g = torch.Generator(device="cuda").manual_seed(t + h + i)
    top, low, zero, more = CODES[fmt]
    cfg = W.LayerConfig("few", e, k, h, i, r or 1, 2.0 * (r or 1), t, 0.0, weight_format=fmt)
    codes = {n: torch.full(s, zero, device="cuda", dtype=torch.int32) for n, s in (("gate", (e, i, h)), ("up", (e, i, h)), ("down", (e, h, i)))}
    codes["gate"][:, :, 0] = top
    codes["up"][:, :, 0] = top
    codes["up"][:, 1::2, 1] = more
    row = torch.arange(h, device="cuda")
    for x in range(e):
        pair = (row * 7 + 3 * x) % (i // 2)
        codes["down"][x, row, 2 * pair] = top
        codes["down"][x, row, 2 * pair + 1] = low
    weights = {n + "_packed": _pack(c) for n, c in codes.items()}
    for n, (rows, cols) in (("gate", (i, h)), ("up", (i, h)), ("down", (h, i))):
        if fmt == "mxfp4":
            s = (torch.randint(124, 126, (e, rows, cols // 32), generator=g, device="cuda").to(torch.int16) << 7).view(BF16)
        else:
            s = (torch.rand(e, rows, cols // 32, generator=g, device="cuda") * 0.2 + 0.1).to(BF16)
        if n != "down":
            s = s[:, ::2].repeat_interleave(2, 1).contiguous()  # of a pair: the same
        weights[n + "_scale"] = s
    lora = {n: torch.zeros(*s, device="cuda") for n, s in cfg.lora_shapes().items()} if r else None
    x = torch.zeros(t, h, device="cuda")
    x[:, 0] = (torch.rand(t, generator=g, device="cuda") + 0.5).to(BF16).float()
    x[:, 1] = x[:, 0] / 32
    x = x.to(BF16)
    ids = torch.rand(t, e, generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    rw = torch.rand(t, k, generator=g, device="cuda") + 0.5
    layer = dev.DeviceLayer.from_tensors(cfg, weights, lora)
    out = layer.decode(x, ids, rw, layer.decode_workspace(t))
    want, bound = torch.zeros(t, h, dtype=F64), torch.zeros(t, h, dtype=F64)
    for a in range(t):
        for b in range(k):
            w = {n: S.weights(weights[n + "_packed"][ids[a, b]].cpu(), weights[n + "_scale"][ids[a, b]].cpu(), fmt) for n in codes}
            v = x[a].double().cpu()
            gv, uv = w["gate"][0] @ v, w["up"][0] @ v
            hv = gv / (1 + torch.exp(-gv)) * uv
            weight = rw[a, b].double().cpu()
            # gate and up are exact but for the product with the scale (two inputs of 8 bits times 5 bits, 1/32 apart: 18 bits, and 24 with
            # the parts that cancel); the sigmoid and the products as elsewhere; h as down reads it to 2^-20
            dh = (16 * R.U * (1 + gv.abs()) + 8 * R.U + 2.0**-20) * hv.abs()
            want[a] += weight * (w["down"][0] @ hv)
            d = w["down"][0].abs()
            bound[a] += weight * (d @ dh)
            if fmt == "mxfp4":  # a sum of down has two products that are not zero
                bound[a] += weight * 16 * R.U * (d @ hv.abs())
            else:
                # 16 s (sum (1 + c / 16) h - 3/2 sum h) over 16 columns, zero weights among them; m is the sum of |h|.  sum h: five levels of
                # additions; times 3/2; eight steps of two products, two roundings each, whose sums stay within 3/2 m:
                # 3/2 (5 + 1 + 16) = 33 roundings of m, times 16 s (a weight is 7 s, a row has two of them)
                m = hv.abs().view(-1, 16).sum(1).repeat_interleave(16)
                bound[a] += weight * 16 * 33 * R.U * (d / 7 @ m) / 2
    bound = 1.1 * bound + 8 * R.U * want.abs()
    R.within("output", out, want, bound + R.UB * (want.abs() + bound))
