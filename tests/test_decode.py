"""GPU: the routed experts for a few tokens against a plain 64-bit implementation and against the
inference forward.  Each case prints its name."""

import pytest

from int4_quantized_moe_amd import workloads as W
from tests import block_reference as R
from tests import step_reference as S

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[decode]", *a, flush=True)


class Case:
    def __init__(self, dev, t, e, k, h, i, r=0, fmt="rawint4", limit=0.0, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cfg = W.LayerConfig("few", e, k, h, i, r or 1, 2.0 * (r or 1), t, limit, weight_format=fmt)
        self.weights = {}
        for name, n, c in (("gate", i, h), ("up", i, h), ("down", h, i)):
            self.weights[name + "_packed"] = torch.randint(0, 256, (e, n, c // 2), generator=g, device="cuda", dtype=torch.uint8)
            if fmt == "mxfp4":
                s = (torch.randint(121, 125, (e, n, c // 32), generator=g, device="cuda").to(torch.int16) << 7).view(BF16)
            else:
                s = (torch.rand(e, n, c // 32, generator=g, device="cuda") * 0.06 + 0.01).to(BF16)
            self.weights[name + "_scale"] = s
        self.lora = None
        if r:
            self.lora = {n: torch.randn(*s, generator=g, device="cuda") * 0.05 for n, s in self.cfg.lora_shapes().items()}
        self.x = (torch.randn(t, h, generator=g, device="cuda") * 0.2).to(BF16)
        self.ids = torch.rand(t, e, generator=g, device="cuda").argsort(1)[:, :k].contiguous()
        self.rw = torch.softmax(torch.randn(t, k, generator=g, device="cuda"), 1)
        self.layer = dev.DeviceLayer.from_tensors(self.cfg, self.weights, self.lora)

    def run(self, **kw):
        return self.layer.decode(self.x, self.ids, self.rw, self.layer.decode_workspace(len(self.x)), **kw)

    def check(self, out):
        want, bound = S.experts(self.x, self.ids, self.rw, self.weights, self.cfg.weight_format, self.cfg.swiglu_limit, self.lora, 2.0)
        R.within("output", out, want, bound + R.UB * (want.abs() + bound))
        # the rounding to bf16 is uniform in at most half a step; everything before it is far below
        rel = S.rel_l2(out, want)
        _say(f"rel_l2 {rel:.2e}")
        assert rel <= R.UB / 3**0.5 + 1e-4


# one token to the most, contractions that end inside a wave's step, experts with several tokens
@pytest.mark.parametrize("t,e,k,h,i", [(1, 4, 2, 32, 32), (1, 8, 8, 256, 128), (2, 6, 3, 160, 224), (3, 5, 2, 96, 512), (4, 4, 1, 288, 64),
                                       (7, 3, 3, 128, 96), (16, 8, 2, 512, 384), (33, 16, 4, 64, 2080), (64, 5, 2, 64, 64),
                                       (64, 16, 16, 32, 32), (5, 2, 2, 1056, 4128)])
@pytest.mark.parametrize("r,fmt,limit", [(0, "rawint4", 0.0), (0, "mxfp4", 1.0), (5, "rawint4", 0.5), (8, "mxfp4", 0.0), (128, "rawint4", 0.0)])
def test_decode(dev, t, e, k, h, i, r, fmt, limit):
    _say(t, e, k, h, i, r, fmt, limit)
    c = Case(dev, t, e, k, h, i, r, fmt, limit, seed=t * h)
    c.check(c.run())


@pytest.mark.parametrize("r", [0, 16])
def test_decode_at_the_full_width(dev, r):
    _say("full width", r)
    c = Case(dev, 3, 12, 8, 7168, 2048, r)
    c.x *= 4
    c.check(c.run())


@pytest.mark.parametrize("t,e,k,h,i,r,fmt", [(2, 2, 2, 16384, 64, 128, "rawint4"), (1, 3, 2, 16352, 32, 0, "mxfp4"), (5, 2, 1, 32, 16416, 3, "mxfp4")])
def test_the_widest_layers(dev, t, e, k, h, i, r, fmt):
    _say("widest", t, e, k, h, i, r, fmt)
    c = Case(dev, t, e, k, h, i, r, fmt, 0.0, seed=t * h)
    c.check(c.run())


@pytest.mark.parametrize("r", [0, 8])
def test_dropped_and_repeated_ids(dev, r):
    """Ids outside the experts add nothing, a token may hold an expert twice, one without any gets zeros, all tokens may share one expert."""
    _say("ids", r)
    c = Case(dev, 9, 6, 4, 128, 160, r)
    c.ids[0] = torch.tensor([2, 2, -1, 2])
    c.ids[1] = -1
    c.ids[2] = torch.tensor([6, 2**40, -(2**40), 5])
    c.ids[3] = torch.tensor([2, 5, 2, 5])
    out = c.run(output=torch.full((9, 128), NAN, dtype=BF16, device="cuda"))
    c.check(out)
    assert not out[1].any()
    c.ids[:] = 3
    c.check(c.run())
    c.ids[:] = -1
    assert not c.run().any()


@pytest.mark.parametrize("h,i,e,fmt", [(128, 160, 6, "rawint4"), (2112, 96, 6, "mxfp4"), (7168, 2048, 8, "rawint4"), (64, 64, 1100, "rawint4")])
@pytest.mark.parametrize("r", [0, 8])
def test_one_token_that_repeats_an_expert(dev, h, i, e, fmt, r):
    _say("one token, repeated", h, i, e, fmt, r)
    c = Case(dev, 1, e, 5, h, i, r, fmt)
    c.ids[0] = torch.tensor([3, 1, 3, 3, 1])
    c.check(c.run())


# above and below what short rows take: slots x intermediate, hidden, rank; intermediates that end inside a workgroup's columns
@pytest.mark.parametrize("t,e,k,h,i", [(2, 6, 3, 160, 2048), (2, 6, 3, 160, 2080), (9, 40, 4, 2048, 352), (9, 40, 4, 2080, 352), (33, 8, 2, 224, 224),
                                       (64, 5, 3, 32, 96)])
@pytest.mark.parametrize("r,fmt,limit", [(0, "rawint4", 0.5), (0, "mxfp4", 0.0), (7, "mxfp4", 1.0), (64, "rawint4", 0.0), (65, "rawint4", 0.0)])
def test_short_rows(dev, t, e, k, h, i, r, fmt, limit):
    _say("short", t, e, k, h, i, r, fmt, limit)
    c = Case(dev, t, e, k, h, i, r, fmt, limit, seed=t + h)
    c.ids[0, 0] = c.ids[0, -1]
    c.ids[-1, 0] = -1
    c.check(c.run())


def test_decode_equals_itself_anywhere(dev):
    """Results repeat bit for bit, from any workspace, and a larger workspace serves fewer tokens."""
    _say("repeat")
    c = Case(dev, 13, 8, 3, 256, 320, 8)
    ws = c.layer.decode_workspace(64)
    outs = []
    for fill in (0x00, 0xFF, 0x7F):
        ws.fill_(fill)
        outs.append(c.layer.decode(c.x, c.ids, c.rw, ws))
    assert all(torch.equal(o, outs[0]) for o in outs) and torch.equal(c.run(), outs[0])
    assert c.layer.decode(c.x[:0], c.ids[:0], c.rw[:0], ws).shape == (0, 256)


def test_decode_is_near_the_inference_forward(dev):
    _say("infer")
    for index in (0, 1):
        cfg, weights, batch = W.make_workload(index)
        layer, b = dev.DeviceLayer(cfg, weights), dev.DeviceBatch(batch)
        a = layer.infer(b.inputs, b.expert_ids, b.route_weights, layer.infer_workspace(b.qlen))
        d = layer.decode(b.inputs, b.expert_ids, b.route_weights, layer.decode_workspace(b.qlen))
        rel = S.rel_l2(d, a)
        _say(cfg.name, f"rel_l2 {rel:.2e}")
        assert rel <= 2 * R.UB / 3**0.5 + 5e-4  # both round to bf16, the inference forward keeps h in fp16


def test_scales_and_inputs_of_any_size(dev):
    """No numeric domain: scales far outside fp16's range, zero ones, inputs of 1e30; not finite ones stay with their token."""
    _say("range")
    c = Case(dev, 4, 3, 1, 64, 64)
    c.ids[:] = torch.tensor([[0], [1], [2], [0]])
    for n in ("gate_scale", "up_scale"):
        c.weights[n][0] *= 2.0**-60
        c.weights[n][1] *= 2.0**40
    c.weights["down_scale"][0] *= 2.0**30
    c.weights["down_scale"][1] *= 2.0**-80
    c.weights["down_scale"][2, :, 1] = 0
    c.x[0] *= 2.0**60
    c.x[3] *= 2.0**60
    c.check(c.run())
    c.x[0, 3] = float("inf")
    out = c.run()
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1:]).all()


def test_decode_in_graphs_and_on_streams(dev):
    """Two captured calls with workspaces of their own, replayed in turn and at once with other inputs, equal the eager ones."""
    _say("graphs")
    cases = [Case(dev, 5, 6, 2, 256, 128, 8, seed=s) for s in (1, 2)]
    graphs, outs, spaces = [], [], []
    side = torch.cuda.Stream()
    for c in cases:
        spaces.append(c.layer.decode_workspace(5))
        outs.append(torch.empty_like(c.x))
        c.layer.decode(c.x, c.ids, c.rw, spaces[-1], output=outs[-1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.layer.decode(c.x, c.ids, c.rw, spaces[-1], output=outs[-1])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        for c in cases:
            c.x.copy_(torch.roll(c.x, i + 1, 0))
            c.ids.copy_(torch.roll(c.ids, 1, 1))
        want = [c.run() for c in cases]
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(NAN)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), i
    with torch.cuda.stream(streams[0]):
        a = cases[0].run()
    b = cases[0].run(stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, want[0])
