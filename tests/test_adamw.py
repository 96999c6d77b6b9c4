"""GPU: AdamW over many tensors, states in 32 and in 8 bits, masters, clipping, skipped steps, against a plain
64-bit implementation.  Each case prints its name."""

import math

import pytest

from tests import block_reference as R
from tests import step_reference as S

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from int4_quantized_moe_amd import device

    return device


def _say(*a):
    print("[adamw]", *a, flush=True)


def _params(seed, sizes, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return {f"t{j}": (torch.randn(n, generator=g) * 0.05).to(dtype).cuda() for j, n in enumerate(sizes)}, g


def _grads(params, g, dtype=F32, size=1e-3):
    return {n: (torch.randn(p.shape, generator=g) * size * 4.0 ** (j % 3)).to(dtype).cuda() for j, (n, p) in enumerate(params.items())}


def _moments(s, states):
    if states == "fp32":
        return s["m"].double().cpu(), s["v"].double().cpu()
    by = lambda x: x.double().repeat_interleave(256)[:s["m"].numel()].cpu()  # noqa: E731
    return s["m"].double().cpu() * by(s["m_scale"]), (s["v"].double().cpu() * by(s["v_scale"])) ** 2


SIZES = [(1,), (3, 256, 255, 257), (4096, 4097, 1, 70001), (5, 0, 9000), tuple(range(1, 80))]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype,grad,master", [(F32, F32, False), (BF16, F32, True), (BF16, BF16, False), (F32, BF16, False)])
@pytest.mark.parametrize("states", ["fp32", "e4m3"])
@pytest.mark.parametrize("clip", [None, 0.01])
def test_steps(dev, sizes, dtype, grad, master, states, clip):
    """Three steps, each against the values that the step before left."""
    _say(sizes if len(sizes) < 9 else len(sizes), dtype, grad, master, states, clip)
    params, g = _params(sum(sizes), sizes, dtype)
    opt = dev.DeviceAdamW(params, lr=2e-3, betas=(0.8, 0.95), eps=1e-7, weight_decay=0.1, states=states, master=master, max_norm=clip,
                          no_decay=("t0",))
    for t in range(1, 4):
        grads = _grads(params, g, grad)
        before = {n: ((opt.state[n]["master"] if master else p).clone(), *_moments(opt.state[n], states)) for n, p in params.items()}
        opt.step(grads, grad_scale=0.5)
        mult = 0.5
        if clip:
            norm = 0.5 * math.sqrt(sum(float(x.double().square().sum()) for x in grads.values()))
            R.within("norm", opt.grad_norm, torch.tensor([norm], dtype=F64), torch.tensor([2 * R.U * norm], dtype=F64))
            mult *= min(1.0, clip / (norm + 1e-6))
        assert int(opt.step_count) == t
        for n, p in params.items():
            s, old = opt.state[n], before[n]
            (e, b), (m, dm), (v, dv) = S.adamw(old[0], grads[n], old[1], old[2], t, lr=2e-3, betas=(0.8, 0.95), eps=1e-7,
                                               weight_decay=0.0 if n == "t0" else 0.1, mult=mult)
            if p.numel() == 0:
                continue
            if master:
                R.within(f"{n} master", s["master"], e, b)
                assert torch.equal(p, s["master"].to(BF16))
            else:
                R.within(f"{n} param", p, e, b + S.rounding(dtype) * (e.abs() + b))
            if states == "fp32":
                R.within(f"{n} m", s["m"], m, dm)
                R.within(f"{n} v", s["v"], v, dv)
            else:
                for key, value, dvalue, root in (("m", m, dm, False), ("v", v.sqrt(), 6 * R.U * v.sqrt(), True)):
                    q, scale, dq, ds = S.e4m3_blocks(value, dvalue, root)
                    R.within(f"{n} {key} scale", s[key + "_scale"], scale, ds)
                    R.within(f"{n} {key} codes", s[key], q, dq)
                    if root:
                        assert ((s[key].float() > 0) == (value.cuda() > 0)).all()


def test_a_norm_that_is_not_finite_changes_nothing(dev):
    _say("skip")
    for states in ("fp32", "e4m3"):
        for value in (float("nan"), float("inf")):
            params, g = _params(3, (300, 5000), F32)
            opt = dev.DeviceAdamW(params, states=states, check_finite=True, step=6)
            opt.step(_grads(params, g))
            kept = {n: [x.clone().view(torch.uint8) for x in (p, *opt.state[n].values())] for n, p in params.items()}
            bad = _grads(params, g)
            bad["t1"][4321] = value
            opt.step(bad)
            assert int(opt.step_count) == 7 and not math.isfinite(float(opt.grad_norm))
            for n, p in params.items():
                assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(kept[n], (p, *opt.state[n].values()))), n
            opt.step(_grads(params, g))
            assert int(opt.step_count) == 8 and math.isfinite(float(opt.grad_norm))


def test_gradients_whose_squares_pass_fp32(dev):
    _say("large")
    params, _ = _params(4, (1000, 2000), F32)
    opt = dev.DeviceAdamW(params, max_norm=1.0)
    grads = {n: torch.full_like(p, 1e30) for n, p in params.items()}
    opt.step(grads)
    norm = 1e30 * math.sqrt(3000)
    assert abs(float(opt.grad_norm) / norm - 1) < 1e-6 and int(opt.step_count) == 1
    m = opt.state["t0"]["m"]
    R.within("m", m, torch.full((1000,), 0.1 * float(torch.tensor(1e30)) / norm, dtype=F64), torch.full((1000,), 1e-6 / 50))


@pytest.mark.parametrize("states", ["fp32", "e4m3"])
def test_resume_learning_rate_and_zero_gradients(dev, states):
    """A run continued from its state equals the run that went on; lr on the GPU equals lr in the call; tensors without a
    gradient and zero blocks stay."""
    _say("resume", states)
    params, g = _params(5, (777, 4096), BF16)
    opt = dev.DeviceAdamW(params, lr=1e-2, states=states, master=True)
    steps = [_grads(params, g) for _ in range(4)]
    for x in steps[:2]:
        opt.step(x)
    again = {n: p.clone() for n, p in params.items()}
    state = {n: {k: x.clone() for k, x in s.items()} for n, s in opt.state.items()}
    other = dev.DeviceAdamW(again, lr=123.0, states=states, master=True, state=state, step=2)
    lr = torch.tensor([1e-2], device="cuda")
    assert float(lr) != 1e-2  # fp32's: the steps differ by its rounding alone
    opt.lr = float(lr)
    for x in steps[2:]:
        opt.step(x)
        other.step(x, lr=lr)
    assert int(other.step_count) == 4
    for n in params:
        assert torch.equal(params[n], again[n])
        assert all(torch.equal(opt.state[n][k].view(torch.uint8), other.state[n][k].view(torch.uint8)) for k in state[n])
    params = {"w": torch.full((600,), 0.5, device="cuda")}
    opt = dev.DeviceAdamW(params, states=states, weight_decay=0.0)
    opt.step({"w": torch.zeros(600, device="cuda")})
    assert (params["w"] == 0.5).all() and not opt.state["w"]["m"].float().any() and not opt.state["w"]["v"].float().any()


def test_small_roots_keep_a_code(dev):
    """A value whose second moment is far below its block's largest is not divided by eps in the next step."""
    _say("small roots")
    g = torch.full((256,), 1e-9, device="cuda")
    g[0] = 1.0
    params = {"w": torch.zeros(256, device="cuda")}
    opt = dev.DeviceAdamW(params, lr=1e-3, states="e4m3", eps=1e-12, weight_decay=0.0)
    opt.step({"w": g})
    assert (opt.state["w"]["v"].float() > 0).all()
    before = params["w"].clone()
    opt.step({"w": g})
    assert ((params["w"] - before).abs() <= 2e-3).all()


def test_a_step_in_a_graph(dev):
    """Replays go on counting, with eager work between them, as eager steps do."""
    _say("graph")
    for states, clip in (("fp32", None), ("e4m3", 0.02)):
        params, g = _params(6, (300, 70000, 4096), F32)
        twin = {n: p.clone() for n, p in params.items()}
        a = dev.DeviceAdamW(params, states=states, max_norm=clip)
        b = dev.DeviceAdamW(twin, states=states, max_norm=clip)
        grads, lr = _grads(params, g), torch.tensor([1e-3], device="cuda")
        a.step(grads, lr=lr)
        b.step(grads, lr=lr)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            a.step(grads, lr=lr)
        for i in range(4):
            for n, x in _grads(params, g).items():
                grads[n].copy_(x)
            lr.mul_(0.5)
            graph.replay()
            b.step(grads, lr=lr)
            torch.cuda.synchronize()
            assert int(a.step_count) == int(b.step_count) == i + 2
            for n in params:
                assert torch.equal(params[n], twin[n]), (i, n)
                assert all(torch.equal(x.view(torch.uint8), b.state[n][k].view(torch.uint8)) for k, x in a.state[n].items())
