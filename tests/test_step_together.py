"""GPU: a block's training step from the operators together: norm, gate, router, experts, the norm behind them with the
residual, their backward to the stream, and AdamW over everything that learns; then tokens decoded through the trained
block.  The stages against 64 bits on the values that reached them, the step in a graph and on another stream.  Each
case prints its name."""

import numpy as np
import pytest

import oracle as O
from int4_quantized_moe_amd import workloads as W
from tests import block_reference as R
from tests import step_reference as S

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LR, EPS = 1e-3, 1e-5


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[together]", *a, flush=True)


def _cpu(t):
    return t.detach().cpu().clone()


class Block:
    """One block whose vectors, gate and adapters learn."""

    def __init__(self, dev, seed=3, stream=F32, states="fp32", max_norm=0.5):
        self.dev, self.cfg = dev, W.CONFIGS[1]
        cfg = self.cfg
        self.weights, self.batch = W.make_weights(cfg, seed), W.make_batch(cfg, seed)
        e, k, h, t = cfg.num_experts, cfg.top_k, cfg.hidden, cfg.qlen
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        base = dev.DeviceLayer(cfg, self.weights)
        packed = {n + p: getattr(base, n + p) for n in ("gate", "up", "down") for p in ("_packed", "_scale")}
        self.lora = {n: v.clone() for n, v in base.lora.items()}
        self.layer = dev.DeviceLayer.from_tensors(cfg, packed, self.lora)
        self.vectors = {"weight": (1 + 0.1 * r(h)).cuda(), "bias": None}
        self.after = {"branch_weight": (1 + 0.1 * r(h)).cuda(), "gate": (0.5 + 0.1 * r(h)).cuda(), "weight": (1 + 0.1 * r(h)).cuda()}
        self.pre = dev.DeviceNorm(h, eps=EPS, weight=self.vectors["weight"])
        self.post = dev.DeviceNorm(h, eps=EPS, scale=0.75, branch_norm=True, **self.after)
        self.gate_weight = (r(e, h) * h**-0.5).to(BF16).cuda()
        self.gate = dev.DeviceLinear(self.gate_weight)
        self.router = dev.DeviceRouter(e, k)
        self.x = r(t, h).to(stream).cuda()
        self.token_gate = torch.rand(t, generator=g).cuda()
        self.dh, self.dy = r(t, h).to(stream).cuda() * 0.1, (r(t, h) * 0.1).to(BF16).cuda()
        new = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.u, self.h, self.y = new(t, h, dtype=BF16), new(t, h, dtype=stream), new(t, h, dtype=BF16)
        self.logits, self.ids, self.rw = new(t, e), new(t, k, dtype=torch.int64), new(t, k)
        self.out, self.dout, self.du, self.du2 = (new(t, h, dtype=BF16) for _ in range(4))
        self.dx1, self.dx, self.dtg = new(t, h, dtype=stream), new(t, h, dtype=stream), new(t)
        self.droute, self.dlogits = new(t, k), new(t, e)
        self.ws, self.wf, self.wb = self.layer.workspace(t), self.gate.workspace(t), self.gate.backward_workspace(t)
        self.wn, self.wd = self.pre.workspace(t), self.layer.decode_workspace(t)
        self.g_pre, self.g_post = self.pre.grad_buffers(), self.post.grad_buffers()
        self.g_lora, self.g_gate = self.layer.grad_buffers(), self.gate.grad_buffers()
        params = {"gate": self.gate_weight, "pre": self.vectors["weight"], **{"post_" + n: v for n, v in self.after.items()}, **self.lora}
        self.grads = {"gate": self.g_gate["weight"], "pre": self.g_pre["weight"], **{"post_" + n: v for n, v in self.g_post.items()},
                      **self.g_lora}
        self.opt = dev.DeviceAdamW(params, lr=LR, states=states, master=True, max_norm=max_norm, no_decay=("pre",))

    def forward(self, **s):
        self.pre.forward(self.x, y=self.u, **s)
        self.gate.forward(self.u, self.wf, output=self.logits, **s)
        self.router.forward(self.logits, expert_ids=self.ids, route_weights=self.rw, **s)
        self.layer.forward(self.u, self.ids, self.rw, self.ws, output=self.out, **s)
        self.post.forward(self.x, branch=self.out, token_gate=self.token_gate, h=self.h, y=self.y, **s)

    def backward(self, **s):
        self.post.backward(self.h, self.wn, self.g_post, branch=self.out, token_gate=self.token_gate, grad_h=self.dh, grad_y=self.dy,
                           grad_x=self.dx1, grad_branch=self.dout, grad_token_gate=self.dtg, **s)
        self.layer.backward(self.u, self.ids, self.rw, self.dout, self.ws, self.g_lora, grad_input=self.du, grad_route=self.droute, **s)
        self.router.backward(self.logits, self.ids, self.droute, grad_logits=self.dlogits, **s)
        self.gate.backward(self.u, self.dlogits, self.wb, self.g_gate, grad_input=self.du2, grad_residual=self.du, **s)
        self.pre.backward(self.x, self.wn, self.g_pre, grad_h=self.dx1, grad_y=self.du2, grad_x=self.dx, **s)

    def run(self, stream=None):
        s = dict(stream=stream)
        self.forward(**s)
        self.backward(**s)
        self.opt.step(self.grads, **s)

    def learned(self):
        return {**self.opt.params, "step": self.opt.step_count, "norm": self.opt.grad_norm,
                **{f"{n}.{k}": v for n, q in self.opt.state.items() for k, v in q.items()}}

    def results(self):
        return {"y": self.y, "h": self.h, "dx": self.dx, "dtg": self.dtg, **self.grads, **{"p." + n: v for n, v in self.learned().items()}}

    def start_over(self, first):
        for n, v in self.learned().items():
            v.copy_(first[n])


def _copy(r):
    torch.cuda.synchronize()
    return {n: t.clone() for n, t in r.items()}


def _same(a, b):
    for n in a:
        assert torch.equal(a[n].contiguous().view(-1).view(torch.uint8), b[n].contiguous().view(-1).view(torch.uint8)), f"{n} differs"


@pytest.mark.parametrize("stream", [F32, BF16])
def test_stages_against_64_bits(dev, stream):
    _say("stages", stream)
    b = Block(dev, stream=stream)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    eps = np.float32(EPS).item()
    _, _, u, du = S.norm_fwd(b.x, eps=eps, weight=b.vectors["weight"])
    R.within("norm", b.u, u, du + R.UB * (u.abs() + du))
    args = dict(eps=eps, scale=0.75, branch_norm=True, **b.after)
    h, dh, y, dy = S.norm_fwd(b.x, b.out, b.token_gate, **args)
    R.within("h", b.h, h, dh + S.rounding(stream) * (h.abs() + dh))
    # (y's norm is of h in 32 bits, before it is rounded)
    R.within("y", b.y, y, dy + R.UB * (y.abs() + dy))
    want = S.norm_bwd(b.h, b.out, b.token_gate, b.dh, b.dy, **args)
    R.within("dout", b.dout, want["branch"][0], want["branch"][1] + R.UB * (want["branch"][0].abs() + want["branch"][1]))
    R.within("dtg", b.dtg, want["token_gate"][0], want["token_gate"][1] + R.U * want["token_gate"][0].abs())
    for n, v in b.g_post.items():
        R.within(n, v, want[n][0], want[n][1] + 2 * R.U * want[n][0].abs())
    want = S.norm_bwd(b.x, None, None, b.dx1, b.du2, eps=eps, weight=b.vectors["weight"])
    R.within("dx", b.dx, want["x"][0], want["x"][1] + S.rounding(stream) * (want["x"][0].abs() + want["x"][1]))
    # the update, from the gradients that reached it
    before = {n: _cpu(p) for n, p in b.opt.params.items()}
    grads = {n: _cpu(v).double() for n, v in b.grads.items()}
    norm = float(sum((v * v).sum() for v in grads.values())) ** 0.5
    b.opt.step(b.grads)
    torch.cuda.synchronize()
    assert abs(float(b.opt.grad_norm) - norm) <= 2 * R.U * norm
    mult = min(1.0, 0.5 / (norm + 1e-6))
    assert mult < 1
    for n, p in b.opt.params.items():
        zero = torch.zeros_like(before[n], dtype=F32)
        (want, bound), (m, dm), (v, dv) = S.adamw(before[n], b.grads[n], zero, zero, 1, lr=LR, weight_decay=0.0 if n == "pre" else 0.01, mult=mult)
        R.within(n, p, want, bound + S.rounding(p.dtype) * (want.abs() + bound))
        R.within(n + " m", b.opt.state[n]["m"].view(m.shape), m, dm)
        R.within(n + " v", b.opt.state[n]["v"].view(v.shape), v, dv)


def test_tokens_decoded_through_the_trained_block(dev):
    """The adapters that the optimizer changed are the ones that decode() reads, and a token's path alone equals its path
    in the batch up to the experts' roundings."""
    _say("decode after training")
    b = Block(dev, seed=4)
    for _ in range(3):
        b.run()
    b.forward()
    u, h, y = b.dev, b.cfg.hidden, None
    packed = {n + p: getattr(b.layer, n + p) for n in ("gate", "up", "down") for p in ("_packed", "_scale")}
    for t in (0, 7, b.cfg.qlen - 1):
        row = slice(t, t + 1)
        _, u = b.pre.forward(b.x[row])
        assert torch.equal(u, b.u[row])
        out = b.layer.decode(u, b.ids[row], b.rw[row], b.wd)
        cfg = b.cfg
        want, bound = S.experts(u, b.ids[row], b.rw[row], packed, limit=cfg.swiglu_limit, lora=b.lora,
                                sc=np.float32(cfg.alpha / cfg.rank).item())
        R.within("decode", out, want, bound + R.UB * (want.abs() + bound))
        rel, cos = O.relative_l2_and_cosine(out.float().cpu().numpy(), b.out[row].float().cpu().numpy())
        # (two forwards that each are within 5e-3 of the oracle)
        assert rel <= 1e-2 and cos >= 0.9999, (t, rel, cos)
        hh, y = b.post.forward(b.x[row], branch=b.out[row], token_gate=b.token_gate[row])
        assert torch.equal(hh, b.h[row]) and torch.equal(y, b.y[row])
        assert not torch.equal(b.lora["up_lora_a"].cpu(), torch.from_numpy(b.weights.lora["up_lora_a"]))


@pytest.mark.parametrize("states", ["fp32", "e4m3"])
def test_step_in_a_graph(dev, states):
    """Captured and replayed with eager steps between: every replay equals the eager step from the same state on the same
    inputs, bit for bit.  Two graphs with buffers of their own do not disturb each other."""
    _say("graph", states)
    a, b = Block(dev, seed=5, states=states), Block(dev, seed=6, stream=BF16, states=states)
    side, graphs = torch.cuda.Stream(), []
    for s in (a, b):
        s.run()
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
            start = _copy(s.learned())
            s.run()
            eager = _copy(s.results())
            s.start_over(start)
            for w in (s.wn, s.ws, s.wb, s.wf):
                w.fill_(0xFF)
            other.replay()
            g.replay()
            torch.cuda.synchronize()
            _same(eager, s.results())


def test_decode_step_in_a_graph(dev):
    """Norm, gate, router, decode and the norm behind it, captured for one token and for several."""
    _say("decode graph")
    b = Block(dev, seed=9)
    for t in (1, 5):
        x, tg = b.x[:t].clone(), b.token_gate[:t].clone()
        wd, wf = b.layer.decode_workspace(t), b.gate.workspace(t)
        keep = {n: torch.zeros_like(v[:t]) for n, v in (("u", b.u), ("logits", b.logits), ("ids", b.ids), ("rw", b.rw), ("out", b.out), ("h", b.h), ("y", b.y))}

        def step():
            b.pre.forward(x, y=keep["u"])
            b.gate.forward(keep["u"], wf, output=keep["logits"])
            b.router.forward(keep["logits"], expert_ids=keep["ids"], route_weights=keep["rw"])
            b.layer.decode(keep["u"], keep["ids"], keep["rw"], wd, output=keep["out"])
            b.post.forward(x, branch=keep["out"], token_gate=tg, h=keep["h"], y=keep["y"])

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for turn in range(3):
            x.copy_(b.x[turn:turn + t] * (1 + turn))
            step()
            eager = _copy(keep)
            for v in keep.values():
                v.zero_()
            wd.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            _same(eager, keep)


def test_step_on_another_stream(dev):
    _say("stream")
    b = Block(dev, seed=7)
    start = _copy(b.learned())
    b.run()
    eager = _copy(b.results())
    side = torch.cuda.Stream()
    for how in ("object", "handle", "current"):
        b.start_over(start)
        for n, v in b.results().items():
            if not n.startswith("p."):
                v.zero_()
        torch.cuda.synchronize()
        if how == "current":
            with torch.cuda.stream(side):
                b.run()
        else:
            b.run(stream=side if how == "object" else side.cuda_stream)
        side.synchronize()
        _same(eager, b.results())
