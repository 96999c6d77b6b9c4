"""GPU: the operators as a layer uses them together: logits, routing, experts,
their backward from an 8-bit checkpoint, and the router's gradients on top of
the experts' grad_input; the same step captured into a HIP graph and replayed,
and on another stream.  Each stage is checked against 64 bits (the experts
against the oracle) on the values that reached it.  Each case prints its name."""

import numpy as np
import pytest

import oracle as O
from int4_quantized_moe_amd import workloads as W
from tests import block_reference as R
from tests.clamp_sides import reference

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
    print("[step]", *a, flush=True)


class Step:
    """One layer step with buffers of its own."""

    def __init__(self, dev, seed=3, fmt="int8", index=1, **router):
        self.dev, self.cfg = dev, W.CONFIGS[index]
        cfg = self.cfg
        self.weights = W.make_weights(cfg, seed)
        self.batch = W.make_batch(cfg, seed)
        self.layer, db = dev.DeviceLayer(cfg, self.weights), dev.DeviceBatch(self.batch)
        self.x, self.dy, t = db.inputs, db.grad_output, db.qlen
        g = torch.Generator().manual_seed(seed)
        gate = (torch.randn(cfg.num_experts, cfg.hidden, generator=g) * cfg.hidden**-0.5).to(BF16).cuda()
        self.bias = (torch.randn(cfg.num_experts, generator=g) * 0.05).cuda()
        self.gate = dev.DeviceLinear(gate)
        self.router_args = dict(score="sigmoid", num_groups=4, top_groups=2, group_top=2, scale=2.5, **router)
        self.router = dev.DeviceRouter(cfg.num_experts, cfg.top_k, bias=self.bias, **self.router_args)
        self.mask = torch.ones(t, dtype=torch.bool, device="cuda")
        self.mask[t - 3:] = False
        self.fmt = fmt
        e, k, h = cfg.num_experts, cfg.top_k, cfg.hidden
        new = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.logits, self.dlogits, self.droute = new(t, e), new(t, e), new(t, k)
        self.ids, self.rw, self.load = new(t, k, dtype=torch.int64), new(t, k), new(e, dtype=torch.int32)
        self.out, self.dx = new(t, h, dtype=BF16), new(t, h, dtype=BF16)
        self.dx_experts = new(t, h, dtype=BF16)
        self.ck = dev.checkpoint8_buffers(t, h, fmt)
        self.grads, self.gate_grads = self.layer.grad_buffers(), self.gate.grad_buffers()
        self.ws = self.layer.checkpoint_workspace(t)
        self.wi = self.layer.infer_workspace(t)
        self.wf, self.wb = self.gate.workspace(t), self.gate.backward_workspace(t)

    def run(self, stream=None):
        s = dict(stream=stream)
        self.gate.forward(self.x, self.wf, output=self.logits, **s)
        self.router.forward(self.logits, token_mask=self.mask, expert_ids=self.ids, route_weights=self.rw,
                            load=self.load, **s)
        self.dev.pack_checkpoint8(self.x, self.fmt, self.ck, **s)
        self.layer.infer(self.x, self.ids, self.rw, self.wi, output=self.out, **s)
        self.layer.backward(self.ck, self.ids, self.rw, self.dy, self.ws, self.grads, grad_input=self.dx_experts,
                            grad_route=self.droute, **s)
        self.router.backward(self.logits, self.ids, self.droute, grad_logits=self.dlogits, **s)
        self.gate.backward(self.ck, self.dlogits, self.wb, self.gate_grads, grad_input=self.dx,
                           grad_residual=self.dx_experts, **s)

    def results(self):
        return {"logits": self.logits, "ids": self.ids, "rw": self.rw, "load": self.load, "out": self.out,
                "dx": self.dx, "droute": self.droute, "dlogits": self.dlogits, "dgate": self.gate_grads["weight"],
                **self.grads}


def _same(a, b):
    for n in a:
        x, y = a[n].contiguous().view(torch.uint8), b[n].contiguous().view(torch.uint8)
        assert torch.equal(x, y), f"{n} differs"


def _copy(r):
    torch.cuda.synchronize()
    return {n: t.clone() for n, t in r.items()}


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_step_against_64_bits(dev, fmt):
    _say("stages", fmt)
    s = Step(dev, fmt=fmt)
    s.run()
    torch.cuda.synchronize()
    cfg = s.cfg
    y, _, b, _ = R.linear(s.x, s.gate.weight)
    R.within("logits", s.logits, y, b + R.U * y.abs())
    l = s.logits.cpu().numpy()
    ids, w, load = R.route(l, cfg.top_k, bias=s.bias.cpu().numpy(), mask=s.mask.cpu().numpy(), **s.router_args)
    assert np.array_equal(s.ids.cpu().numpy(), ids) and np.array_equal(s.load.cpu().numpy(), load)
    R.within("route weights", s.rw, w, 2 * R.route_precision(l)[:, None] * np.abs(w))
    rows = dev.unpack_checkpoint8(s.ck)
    R.within("checkpoint", rows, R.checkpoint(s.x.float().cpu().numpy(), fmt), np.zeros(tuple(s.x.shape)))

    rw = s.rw.cpu().numpy()
    fwd = O.moe(cfg, s.weights, s.batch.inputs, ids, rw, s.batch.grad_output)
    rel, cos = O.relative_l2_and_cosine(s.out.float().cpu().numpy(), fwd["out"])
    assert rel <= 5e-3 and cos >= 0.9999, (rel, cos)
    # the backward's pre-activations are those of the unpacked rows
    ws = s.layer.workspace(len(rows))
    s.layer.forward(rows, s.ids, s.rw, ws)
    pre = tuple(t.cpu().numpy() for t in s.layer.saved_preactivations(len(rows), ws))
    from int4_quantized_moe_amd.device import bf16_bits

    ref = reference(cfg, s.weights, bf16_bits(rows), ids, rw, s.batch.grad_output, pre, _say)
    for name, a, e, bar in [("dX of the experts", s.dx_experts.float().cpu().numpy(), ref["dx"], 5e-3),
                            ("dRoute", s.droute.cpu().numpy(), ref["droute"], 3e-2)] + \
                           [(n, s.grads[n].cpu().numpy(), ref["grads"][n], 5e-3) for n in O.LORA_NAMES]:
        rel, cos = O.relative_l2_and_cosine(a, e)
        _say(f"{name}: rel_l2={rel:.2e} cos={cos:.6f}")
        assert rel <= bar and cos >= 0.995, name

    want, bound = R.route_bwd(l, ids, s.droute.cpu().numpy(), score="sigmoid", renormalize=True, scale=2.5)
    R.within("dlogits", s.dlogits, want, bound + R.U * np.abs(want) + 2.0**-126)
    assert not s.dlogits[~s.mask].any()
    want, bound = R.linear_bwd(rows, s.gate.weight, s.dlogits, grad_residual=s.dx_experts)
    R.within("dx", s.dx, want["dx"], bound["dx"] + R.UB * want["dx"].abs())
    R.within("dgate", s.gate_grads["weight"], want["dw"], bound["dw"] + 2 * R.U * want["dw"].abs())


def test_step_in_a_graph(dev):
    """Captured and replayed, with eager work and other inputs between the replays: every replay equals the
    eager step on the same inputs, bit for bit.  Two graphs with buffers of their own do not disturb each other."""
    _say("graph")
    a, b = Step(dev, seed=5), Step(dev, seed=6)
    side = torch.cuda.Stream()
    graphs = []
    for s in (a, b):
        s.run()  # (first calls outside the capture)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.run()
        graphs.append(g)
    first = a.x.clone()
    for turn in range(3):
        for s, g, other in ((a, graphs[0], graphs[1]), (b, graphs[1], graphs[0])):
            if s is a:
                a.x.copy_(torch.roll(first, turn, 0) * (turn + 1))
            s.run()
            eager = _copy(s.results())
            for t in s.results().values():
                t.zero_()
            s.ws.fill_(0xFF), s.wb.fill_(0xFF), s.wf.fill_(0xFF)
            other.replay()
            g.replay()
            torch.cuda.synchronize()
            _same(eager, s.results())


def test_step_on_another_stream(dev):
    _say("stream")
    s = Step(dev, seed=7)
    s.run()
    eager = _copy(s.results())
    for t in s.results().values():
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s.run(stream=side)
    side.synchronize()
    _same(eager, s.results())
    with torch.cuda.stream(side):  # the current stream
        for t in s.results().values():
            t.zero_()
        s.run()
    side.synchronize()
    _same(eager, s.results())


def test_outputs_made_by_the_calls(dev):
    """Without given buffers, and with a stream given as an object or a handle."""
    _say("made outputs")
    s = Step(dev, seed=8)
    s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        logits = s.gate.forward(s.x, s.wf, dtype=F32, stream=stream)
        ids, rw = s.router.forward(logits, token_mask=s.mask, stream=stream)
        ck = dev.pack_checkpoint8(s.x, "int8", stream=stream)
        rows = dev.unpack_checkpoint8(ck, stream=stream)
        dl = s.router.backward(logits, ids, s.droute, stream=stream)
        dx = s.gate.backward(ck, dl, s.wb, {}, grad_residual=s.dx_experts, stream=stream)
        torch.cuda.synchronize()
        for x, y in ((logits, s.logits), (ids, s.ids), (rw, s.rw), (ck.codes, s.ck.codes), (dl, s.dlogits), (dx, s.dx),
                     (rows, dev.unpack_checkpoint8(s.ck))):
            assert torch.equal(x, y)


def test_balance_over_steps(dev):
    """The bias's rule on the counted load evens out a skewed router (a known direction: every expert above the
    mean load loses bias, every one below gains)."""
    _say("balance")
    e, k, t = 16, 2, 512
    g = torch.Generator().manual_seed(1)
    logits = (torch.randn(t, e, generator=g) + torch.linspace(1, -1, e)).cuda()
    router = dev.DeviceRouter(e, k, score="sigmoid", bias=torch.zeros(e, device="cuda"))
    load = torch.zeros(e, dtype=torch.int32, device="cuda")
    for _ in range(5):
        before = router.bias.clone()
        router.forward(logits, load=load)
        router.update_bias(load, 0.01)
        step = torch.sign(load.sum() - load.long() * e).float() * np.float32(0.01)
        assert torch.equal(router.bias, before + step)
    assert int(load.sum()) == t * k
