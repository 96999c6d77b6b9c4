"""What completes a step, on the CPU: the library exports what include/kt_step.h declares, the binding's constants
and structs are the header's, and every entry point and class refuses wrong arguments before any GPU work."""

import ctypes
import os
import re

import pytest

import int4_quantized_moe_amd as kt
from int4_quantized_moe_amd import _lib, workloads

from .conftest import ROOT

torch = pytest.importorskip("torch")
from int4_quantized_moe_amd import device  # noqa: E402

HEADER = open(os.path.join(ROOT, "include", "kt_step.h")).read()
FAKE = 1 << 20  # a non-null, 256-aligned address; never dereferenced by the host checks
NAN, INF = float("nan"), float("inf")


def test_library_exports_every_declared_symbol():
    names = sorted(set(re.findall(r"^(?:int|size_t) (kt_\w+)\(", HEADER, re.M)))
    assert len(names) == 7
    bound = _lib.load_library()
    for name in names:
        assert getattr(bound, name).argtypes is not None and hasattr(kt, name), name


def test_constants_and_structs_match_the_header():
    seen = 0
    for name, value in re.findall(r"#define (KT_\w+) (\d+)", HEADER):
        assert getattr(_lib, name) == int(value), name
        seen += 1
    assert seen == 10
    for struct in ("kt_norm", "kt_adamw", "kt_adamw_tensor"):
        body = re.search(r"typedef struct %s \{(.*?)\}" % struct, HEADER, re.S).group(1)
        names = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
        assert names == [n for n, _ in getattr(_lib, struct)._fields_], struct


def _fails(rc, message, code=kt.KT_RAWINT4_EINVAL):
    assert rc == code, (rc, kt.kt_rawint4_last_error())
    assert message in kt.kt_rawint4_last_error(), kt.kt_rawint4_last_error()


# ---------------------------------------------------------------- norms


def _norm(**over):
    args = dict(hidden=64, kind=0, stream_type=1, branch_norm=1, eps=1e-6, scale=1.0, weight=FAKE, bias=None, branch_weight=FAKE,
                branch_bias=None, gate=None)
    args.update(over)
    return kt.kt_norm(*args.values())


@pytest.mark.parametrize("over,message", [
    (dict(hidden=0), "hidden"), (dict(hidden=16385), "hidden"), (dict(hidden=-1), "hidden"), (dict(kind=2), "kind"),
    (dict(stream_type=2), "stream_type"), (dict(branch_norm=2), "branch_norm"), (dict(eps=-1.0), "eps"), (dict(eps=NAN), "eps"),
    (dict(scale=INF), "scale"), (dict(branch_norm=0), "need branch_norm"), (dict(weight=FAKE + 8), "16-byte"),
    (dict(gate=FAKE + 4), "16-byte")])
def test_invalid_norms_are_refused(over, message):
    lib, n = _lib.load_library(), _norm(**over)
    _fails(lib.kt_norm_fwd(ctypes.byref(n), 4, FAKE, FAKE, None, FAKE, FAKE, None), message)
    _fails(lib.kt_norm_bwd(ctypes.byref(n), 4, *[FAKE] * 7, *[None] * 6, 0, 1.0, FAKE, 1 << 30, None), message)
    assert lib.kt_norm_bwd_workspace_bytes(ctypes.byref(n), 4) == 0


def test_norm_arguments_are_refused():
    lib, n = _lib.load_library(), _norm()
    fwd = lambda t=4, x=FAKE, b=FAKE, tg=None, h=FAKE, y=FAKE, n=n: lib.kt_norm_fwd(ctypes.byref(n) if n else None, t, x, b, tg, h, y, None)  # noqa: E731
    _fails(fwd(n=None), "norm is NULL")
    _fails(fwd(t=-1), "tokens")
    _fails(fwd(t=(1 << 23) + 1), "tokens")
    _fails(fwd(x=None), "x must be")
    _fails(fwd(h=None, y=None), "one of h and y")
    _fails(fwd(b=None), "without a branch")
    _fails(fwd(b=None, h=None, tg=FAKE), "without a branch")
    for k in "xbhy":
        _fails(fwd(**{k: FAKE + 8}), "aligned")
    _fails(fwd(tg=FAKE + 2), "aligned")
    assert fwd(t=0, x=None, b=None, h=None, y=None) == 0

    def bwd(t=4, h=FAKE, b=FAKE, tg=FAKE, gh=FAKE, gy=FAKE, gx=FAKE, gb=FAKE, gtg=FAKE, w=FAKE, c=FAKE, bw=FAKE, bc=FAKE, g=FAKE, acc=0,
            scale=1.0, ws=FAKE, size=1 << 30, n=n):
        return lib.kt_norm_bwd(ctypes.byref(n), t, h, b, tg, gh, gy, gx, gb, gtg, w, c, bw, bc, g, acc, scale, ws, size, None)

    _fails(bwd(t=-1), "tokens")
    _fails(bwd(h=None), "h must be")
    _fails(bwd(gh=None, gy=None), "one of grad_h and grad_y")
    _fails(bwd(gy=None), "need grad_y")
    _fails(bwd(b=None), "need a branch")
    _fails(bwd(tg=None), "needs token_gate")
    _fails(bwd(acc=2), "accumulate")
    _fails(bwd(scale=NAN), "grad_scale")
    _fails(bwd(n=_norm(branch_norm=0, branch_weight=None)), "need branch_norm")
    for k in ("h", "b", "gh", "gy", "gx", "gb", "w", "c", "bw", "bc", "g"):
        _fails(bwd(**{k: FAKE + 8}), "aligned")
    for k in ("tg", "gtg"):
        _fails(bwd(**{k: FAKE + 2}), "aligned")
    _fails(bwd(ws=None), "workspace")
    _fails(bwd(ws=FAKE + 16), "256")
    need = lib.kt_norm_bwd_workspace_bytes(ctypes.byref(n), 4)
    _fails(bwd(size=need - 1), "smaller", kt.KT_RAWINT4_EWORKSPACE)


def test_sizes_grow_with_the_tokens():
    lib = _lib.load_library()
    for h in (1, 64, 511, 512, 513, 7168, 16384):
        n, last = _norm(hidden=h), 0
        for t in [*range(0, 700), *range(700, 5000, 37), 1 << 16, 1 << 23]:
            size = lib.kt_norm_bwd_workspace_bytes(ctypes.byref(n), t)
            assert size >= last and size % 256 == 0
            last = size
    last = 0
    for t in range(0, 200):
        size = kt.kt_adamw_workspace_bytes(t)
        assert size >= last and size % 256 == 0
        last = size
    for r in (0, 16):
        layer, last = _layer(rank=r), 0
        for t in range(0, 65):
            size = kt.kt_moe_decode_workspace_bytes(layer, t)
            assert size >= last and size % 256 == 0
            last = size


def test_norm_class_refuses(monkeypatch):
    with pytest.raises(ValueError, match="kind"):
        device.DeviceNorm(8, "batch")
    for bad in (torch.zeros(7), torch.zeros(8, dtype=torch.float64), torch.zeros(16)[::2]):
        with pytest.raises(ValueError, match="gate"):
            device.DeviceNorm(8, gate=bad)
    n = device.DeviceNorm(8, weight=torch.ones(8), branch_norm=True)
    x, b = torch.zeros(3, 8), torch.zeros(3, 8, dtype=torch.bfloat16)
    for args, kw, word in (((x.double(),), {}, "x"), ((torch.zeros(8),), {}, "tokens"), ((torch.zeros(3, 7),), {}, "shape"),
                           ((torch.zeros(8, 3).t(),), {}, "contiguous"), ((x.to("meta"),), {}, "on cpu"), ((x,), dict(branch=x), "branch"),
                           ((x,), dict(branch=b[:2]), "branch"), ((x,), dict(branch=b, token_gate=torch.zeros(2)), "token_gate"),
                           ((x,), dict(branch=b, h=b), "h must be"), ((x,), dict(y=x), "y must be"), ((x,), dict(h=x), "branch"),
                           ((x,), dict(token_gate=torch.zeros(3)), "branch"), ((x,), {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            n.forward(*args, **kw)
    ws = torch.zeros(1, dtype=torch.uint8)
    for grads, kw, word in (({}, dict(grad_h=b), "grad_h"), ({}, dict(grad_y=x), "grad_y"), ({}, dict(grad_x=b), "grad_x"),
                            ({}, dict(grad_branch=x), "grad_branch"), ({}, dict(grad_token_gate=x), "grad_token_gate"),
                            ({"weight": torch.zeros(7)}, {}, "weight"), ({"scale": torch.zeros(8)}, {}, "no place"), ({}, {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            n.backward(x, ws, grads, **kw)
    with pytest.raises(kt.KtRawInt4Error, match="hidden"):
        device.DeviceNorm(16385, branch_norm=False).workspace(4, device="cpu")
    assert set(n.grad_buffers()) == {"weight"} and n.grad_buffers(fill=2.0)["weight"].sum() == 16


# ---------------------------------------------------------------- AdamW


def _hyper(**over):
    args = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_norm=0.0, grad_scale=1.0, state_format=0)
    args.update(over)
    return kt.kt_adamw(*args.values())


def _tensor(**over):
    args = dict(count=8, param_type=1, grad_type=1, decay=1, param=FAKE, master=None, grad=FAKE, m=FAKE, v=FAKE, m_scale=None, v_scale=None)
    args.update(over)
    return kt.kt_adamw_tensor(*args.values())


def _step(hyper, tensors, n=None, step=FAKE, norm=None, lr=None, ws=FAKE, size=1 << 30):
    array = (kt.kt_adamw_tensor * max(1, len(tensors)))(*tensors)
    return _lib.load_library().kt_adamw_step(ctypes.byref(hyper) if hyper else None, array, len(tensors) if n is None else n, step, norm, lr, ws,
                                             size, None)


@pytest.mark.parametrize("over,message", [
    (dict(lr=NAN), "lr"), (dict(weight_decay=INF), "weight_decay"), (dict(grad_scale=NAN), "grad_scale"), (dict(beta1=1.0), "beta1"),
    (dict(beta1=-0.1), "beta1"), (dict(beta2=1.0), "beta2"), (dict(beta2=NAN), "beta2"), (dict(eps=-1e-8), "eps"), (dict(eps=INF), "eps"),
    (dict(max_norm=-1.0), "max_norm"), (dict(max_norm=NAN), "max_norm"), (dict(max_norm=1.0), "needs grad_norm"), (dict(state_format=2), "state_format")])
def test_invalid_steps_are_refused(over, message):
    _fails(_step(_hyper(**over), [_tensor()]), message)


@pytest.mark.parametrize("over,message", [
    (dict(count=-1), "count"), (dict(count=(1 << 36) + 1), "count"), (dict(param_type=2), "param_type"), (dict(grad_type=-1), "grad_type"),
    (dict(decay=2), "decay"), (dict(master=FAKE), "master"), (dict(param=None), "non-NULL"), (dict(grad=None), "non-NULL"),
    (dict(m=None), "non-NULL"), (dict(v=None), "non-NULL"), (dict(m_scale=FAKE), "must be NULL"), (dict(v_scale=FAKE), "must be NULL"),
    (dict(param=FAKE + 8), "aligned"), (dict(grad=FAKE + 4), "aligned"), (dict(m=FAKE + 8), "aligned"), (dict(v=FAKE + 2), "aligned")])
def test_invalid_tensors_are_refused(over, message):
    _fails(_step(_hyper(), [_tensor(), _tensor(**over)]), message)


def test_step_arguments_are_refused():
    _fails(_step(None, [_tensor()]), "hyper is NULL")
    _fails(_step(_hyper(), [_tensor()], n=-1), "num_tensors")
    _fails(_step(_hyper(), [_tensor()], n=65537), "num_tensors")
    _fails(_lib.load_library().kt_adamw_step(ctypes.byref(_hyper()), None, 1, FAKE, None, None, FAKE, 1 << 30, None), "tensors must be")
    _fails(_step(_hyper(), [_tensor()], step=None), "step")
    _fails(_step(_hyper(), [_tensor()], step=FAKE + 4), "step")
    _fails(_step(_hyper(), [_tensor()], norm=FAKE + 2), "aligned")
    _fails(_step(_hyper(), [_tensor()], lr=FAKE + 2), "aligned")
    _fails(_step(_hyper(state_format=1), [_tensor()]), "8-bit states need")
    _fails(_step(_hyper(state_format=1), [_tensor(m_scale=FAKE, v_scale=FAKE + 4)]), "aligned")
    _fails(_step(_hyper(), [_tensor()], ws=None), "workspace")
    _fails(_step(_hyper(), [_tensor()], size=kt.kt_adamw_workspace_bytes(1) - 1), "smaller", kt.KT_RAWINT4_EWORKSPACE)
    assert _lib.load_library().kt_adamw_workspace_bytes(-1) == 0 and "num_tensors" in kt.kt_rawint4_last_error()


def test_adamw_class_refuses():
    w = {"a": torch.zeros(300), "b": torch.zeros(4, 4, dtype=torch.bfloat16)}
    new = lambda p=w, **kw: device.DeviceAdamW(p, **kw)  # noqa: E731
    for p, kw, word in ((w, dict(states="int8"), "states"), ({}, {}, "params"), ({"a": torch.zeros(3, dtype=torch.float64)}, {}, "a must be"),
                        ({"a": torch.zeros(4, 4).t()[1:]}, {}, "contiguous"), ({**w, "c": torch.zeros(3, device="meta")}, {}, "must be on"),
                        (w, dict(no_decay=("x",)), "no_decay"), (w, dict(state={"a": {"m": torch.zeros(299)}}), "shape"),
                        (w, dict(state={"a": {"m": torch.zeros(300).bfloat16()}}), "float32"),
                        (w, dict(state={"a": {"m_scale": torch.zeros(2)}}), "no place"),
                        (w, dict(states="e4m3", state={"a": {"m_scale": torch.zeros(1)}}), "shape"),
                        (w, dict(step=torch.zeros(1)), "step"), (w, dict(step=torch.zeros(2, dtype=torch.int64)), "step")):
        with pytest.raises(ValueError, match=word):
            new(p, **kw)
    o = new(states="e4m3", master=True, step=3)
    assert int(o.step_count) == 3 and o.grad_norm is None and set(o.state["a"]) == {"m", "v", "m_scale", "v_scale"}
    assert o.state["b"]["master"].shape == (4, 4) and o.state["a"]["m_scale"].shape == (2,)
    grads = {"a": torch.zeros(300), "b": torch.zeros(4, 4)}
    for g, kw, word in (({"a": grads["a"]}, {}, "no 'b'"), ({**grads, "b": torch.zeros(4, 5)}, {}, "shape"),
                        ({**grads, "a": grads["a"].double()}, {}, "float32 or"), (grads, dict(lr=torch.zeros(2)), "lr"), (grads, {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            o.step(g, **kw)


# ---------------------------------------------------------------- experts


def _layer(e=8, k=2, h=64, i=96, rank=4, limit=0.0, fmt=0, lora=FAKE):
    p = [FAKE] * 6 + [lora if rank else None] * 6
    return kt.make_layer(e, k, h, i, rank or 1, 1.0, limit, *p, weight_format=fmt)


def test_decode_arguments_are_refused():
    lib = _lib.load_library()

    def call(layer=_layer(), t=4, x=FAKE, ids=FAKE, rw=FAKE, o=FAKE, ws=FAKE, size=1 << 30):
        return lib.kt_moe_decode(ctypes.byref(layer) if layer else None, t, x, ids, rw, o, ws, size, None)

    _fails(call(layer=None), "layer is NULL")
    _fails(call(layer=_layer(h=48)), "hidden")
    _fails(call(layer=_layer(h=16416)), "16384")
    _fails(call(layer=_layer(k=9)), "top_k")
    _fails(call(layer=_layer(fmt=2)), "weight_format")
    _fails(call(layer=_layer(limit=NAN)), "swiglu_limit")
    partial = _layer()
    partial.up_lora_b = None
    _fails(call(layer=partial), "NULL")
    _fails(call(t=-1), "qlen")
    _fails(call(t=65), "64 tokens")
    _fails(call(layer=_layer(e=100, k=17), t=61), "1024 token-slots")
    for k in ("x", "ids", "rw", "o"):
        _fails(call(**{k: None}), "non-NULL")
    for k, by in (("x", 8), ("ids", 4), ("rw", 2), ("o", 1)):
        _fails(call(**{k: FAKE + by}), "aligned")
    _fails(call(ws=None), "workspace")
    _fails(call(size=kt.kt_moe_decode_workspace_bytes(_layer(), 4) - 1), "smaller", kt.KT_RAWINT4_EWORKSPACE)
    assert lib.kt_moe_decode_workspace_bytes(ctypes.byref(_layer()), 65) == 0
    with pytest.raises(kt.KtRawInt4Error, match="64 tokens"):
        kt.kt_moe_decode_workspace_bytes(_layer(), 65)
    assert call(t=0, x=None, ids=None, rw=None, o=None, ws=None, size=0) == 0


def test_layer_on_tensors_and_decode_refuse():
    cfg = workloads.LayerConfig("few", 4, 2, 64, 32, 8, 8.0, 5, 0.0)
    w = {}
    for name, n, k in (("gate", 32, 64), ("up", 32, 64), ("down", 64, 32)):
        w[name + "_packed"] = torch.zeros(4, n, k // 2, dtype=torch.uint8)
        w[name + "_scale"] = torch.zeros(4, n, k // 32, dtype=torch.bfloat16)
    lora = {n: torch.zeros(s) for n, s in cfg.lora_shapes().items()}
    for name, bad in (("up_packed", w["up_packed"][:3]), ("down_scale", w["down_scale"].float()), ("gate_packed", w["gate_packed"].char()),
                      ("up_scale", w["up_scale"].to("meta"))):
        with pytest.raises(ValueError, match=name):
            device.DeviceLayer.from_tensors(cfg, {**w, name: bad}, lora)
    with pytest.raises(ValueError, match="up_lora_a"):
        device.DeviceLayer.from_tensors(cfg, w, {n: t for n, t in lora.items() if n != "up_lora_a"})
    with pytest.raises(ValueError, match="down_lora_b"):
        device.DeviceLayer.from_tensors(cfg, w, {**lora, "down_lora_b": lora["down_lora_b"].double()})
    layer = device.DeviceLayer.from_tensors(cfg, w, lora)
    x, ids, rw = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)
    ws = torch.zeros(1, dtype=torch.uint8)
    for args, kw, word in (((x.float(), ids, rw), {}, "inputs"), ((x[0], ids, rw), {}, "tokens"), ((x[:, :32].contiguous(), ids, rw), {}, "inputs"),
                           ((x, ids.int(), rw), {}, "expert_ids"), ((x, ids[:2], rw), {}, "expert_ids"), ((x, ids, rw.double()), {}, "route_weights"),
                           ((x, ids, rw), dict(output=x.float()), "output"), ((x, ids, rw), {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            layer.decode(*args, ws, **kw)
