"""GPU: norms, AdamW and the experts for a few tokens write nothing outside their outputs and workspaces, and reach
values behind 2^31.  Each case prints its name first."""

import pytest

from tests.test_block_memory import Buffers
from int4_quantized_moe_amd import workloads as W

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
    print("[step memory]", *a, flush=True)


def _rand(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _into(b, name, value):
    t = b.new(name, tuple(value.shape), value.dtype)
    t.copy_(value)
    return t


@pytest.mark.parametrize("t,h", [(1, 1), (3, 7), (5, 9), (37, 500), (259, 513), (300, 2049), (17, 4100), (9, 7168), (5, 8193), (3, 16383)])
@pytest.mark.parametrize("kind,stream,post", [("rms", BF16, True), ("layer", F32, True), ("layer", BF16, False)])
def test_norms_keep_to_their_buffers(dev, t, h, kind, stream, post):
    _say("norm", t, h, kind, stream, post)
    b = Buffers()
    names = ["weight", "bias", "gate"] + (["branch_weight", "branch_bias"] if post else [])
    v = {n: _rand(i, h) for i, n in enumerate(names)}
    x, branch, tg = _rand(9, t, h, dtype=stream), _rand(10, t, h, dtype=BF16), _rand(11, t)
    norm = dev.DeviceNorm(h, kind, branch_norm=post, **v)
    plain = norm.forward(x, branch=branch, token_gate=tg)
    out = norm.forward(x, branch=branch, token_gate=tg, h=b.new("h", (t, h), stream), y=b.new("y", (t, h), BF16))
    gh, gy = _rand(12, t, h, dtype=stream), _rand(13, t, h, dtype=BF16)
    ws = b.new("workspace", (norm.workspace(t).numel(),), torch.uint8)
    grads = {n: b.new("d " + n, (h,), F32) for n in v}
    dtg = b.new("d token_gate", (t,), F32)
    args = dict(branch=branch, token_gate=tg, grad_h=gh, grad_y=gy)
    norm.backward(out[0], ws, grads, grad_x=b.new("dx", (t, h), stream), grad_branch=b.new("dbranch", (t, h), BF16), grad_token_gate=dtg, **args)
    b.check()
    assert torch.equal(out[0], plain[0]) and torch.equal(out[1], plain[1])
    own = norm.grad_buffers()
    norm.backward(out[0], norm.workspace(t), own, grad_token_gate=torch.empty_like(dtg), **args)
    assert all(torch.equal(own[n], grads[n]) for n in own)


@pytest.mark.parametrize("sizes", [(1, 2, 3, 255, 256, 257), (4095, 4096, 4097, 1023), (5, 12289, 8191)])
@pytest.mark.parametrize("dtype,grad,master,states", [(F32, F32, False, "fp32"), (BF16, BF16, False, "fp32"), (BF16, F32, True, "e4m3"),
                                                      (F32, BF16, False, "e4m3"), (BF16, BF16, True, "fp32")])
def test_steps_keep_to_their_tensors(dev, sizes, dtype, grad, master, states):
    _say("adamw", sizes, dtype, grad, master, states)
    b = Buffers()
    params, grads, state = {}, {}, {}
    for i, n in enumerate(sizes):
        name = f"p{i}"
        params[name] = _into(b, name, _rand(i, n).to(dtype))
        grads[name] = _rand(50 + i, n).to(grad)
        state[name] = s = {}
        if states == "e4m3":
            for k in ("m", "v"):
                s[k] = b.new(f"{name}.{k}", (n,), torch.uint8).zero_().view(torch.float8_e4m3fn)
                s[k + "_scale"] = b.new(f"{name}.{k}_scale", (-(-n // 256),), F32).zero_()
        else:
            for k in ("m", "v"):
                s[k] = b.new(f"{name}.{k}", (n,), F32).zero_()
        if master:
            s["master"] = _into(b, name + ".master", params[name].float())
    own = {n: p.clone() for n, p in params.items()}
    opts = [dev.DeviceAdamW(params, states=states, master=master, max_norm=1.0, state=state),
            dev.DeviceAdamW(own, states=states, master=master, max_norm=1.0)]
    opts[0]._workspace = b.new("workspace", tuple(opts[0]._workspace.shape), torch.uint8)
    for _ in range(2):
        for o in opts:
            o.step(grads)
    b.check()
    assert all(torch.equal(params[n], own[n]) for n in own)


@pytest.mark.parametrize("t,e,k,h,i,r,fmt", [(1, 1, 1, 32, 32, 0, "rawint4"), (3, 5, 2, 160, 224, 8, "mxfp4"), (7, 4, 4, 96, 1056, 5, "rawint4"),
                                             (64, 9, 3, 544, 96, 16, "rawint4"), (2, 300, 10, 1024, 544, 0, "mxfp4")])
def test_decode_keeps_to_its_buffers(dev, t, e, k, h, i, r, fmt):
    _say("decode", t, e, k, h, i, r, fmt)
    b = Buffers()
    cfg = W.LayerConfig("memory", e, k, h, i, max(r, 1), 2.0, t, 3.0, weight_format=fmt)
    w, batch = W.make_weights(cfg, 5), W.make_batch(cfg, 5)
    whole, db = dev.DeviceLayer(cfg, w), dev.DeviceBatch(batch)
    names = [n + p for n in ("gate", "up", "down") for p in ("_packed", "_scale")]
    lora = {n: _into(b, n, v) for n, v in whole.lora.items()} if r else None
    layer = dev.DeviceLayer.from_tensors(cfg, {n: _into(b, n, getattr(whole, n)) for n in names}, lora)
    ws = b.new("workspace", (layer.decode_workspace(t).numel(),), torch.uint8)
    out = layer.decode(_into(b, "x", db.inputs), _into(b, "ids", db.expert_ids), _into(b, "weights", db.route_weights), ws,
                       output=b.new("out", (t, h), BF16))
    b.check()
    if r:
        assert torch.equal(out, whole.decode(db.inputs, db.expert_ids, db.route_weights, whole.decode_workspace(t)))


def test_rows_behind_two_to_the_31(dev):
    """The last rows of a batch of 2.3e9 values equal those rows alone, forward and backward."""
    _say("long batch")
    t, h, n = 140_001, 16_384, 40
    assert (t - n) * h > 2**31
    norm = dev.DeviceNorm(h, weight=_rand(0, h), branch_norm=True, branch_weight=_rand(1, h))
    x, branch = torch.zeros(t, h, dtype=BF16, device="cuda"), torch.zeros(t, h, dtype=BF16, device="cuda")
    x[-n:], branch[-n:] = _rand(2, n, h, dtype=BF16), _rand(3, n, h, dtype=BF16)
    hh, y = norm.forward(x, branch=branch)
    h1, y1 = norm.forward(x[-n:].clone(), branch=branch[-n:].clone())
    assert torch.equal(hh[-n:], h1) and torch.equal(y[-n:], y1) and not hh[:-n].any() and not y[:-n].any()
    del y
    gy = torch.zeros(t, h, dtype=BF16, device="cuda")
    gy[-n:] = _rand(4, n, h, dtype=BF16)
    gx, gb = norm.backward(hh, norm.workspace(t), norm.grad_buffers(), branch=branch, grad_y=gy)
    a, c = norm.backward(h1, norm.workspace(n), norm.grad_buffers(), branch=branch[-n:].clone(), grad_y=gy[-n:].clone())
    assert torch.equal(gx[-n:], a) and torch.equal(gb[-n:], c) and not gx[:-n].any()


@pytest.mark.parametrize("states", ["fp32", "e4m3"])
def test_values_behind_two_to_the_31(dev, states):
    """The tail of a tensor of 2.2e9 values is updated as the tail alone is."""
    _say("long tensor", states)
    n, tail = 2**31 + 4096 * 7 + 513, 4096 * 2 + 513
    assert (n - tail) % 256 == 0
    p, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    p[-tail:], g[-tail:] = _rand(1, tail, dtype=BF16), _rand(2, tail, dtype=BF16)
    one = {"p": p[-tail:].clone()}
    big = dev.DeviceAdamW({"p": p}, states=states, max_norm=1.0)
    small = dev.DeviceAdamW(one, states=states, max_norm=1.0)
    for _ in range(2):
        big.step({"p": g})
        small.step({"p": g[-tail:].clone()})
    assert torch.equal(p[-tail:], one["p"]) and torch.equal(big.grad_norm, small.grad_norm)
    assert not p[:-tail].any()
    for k in ("m", "v"):
        assert torch.equal(big.state["p"][k][-tail:].view(torch.uint8), small.state["p"][k].view(torch.uint8))
