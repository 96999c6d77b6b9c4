"""The operators around the experts on the CPU: the library exports what
include/kt_block.h declares, the binding's constants are the header's, and
every entry point and class refuses wrong arguments before any GPU work."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

import int4_quantized_moe_amd as kt
from int4_quantized_moe_amd import _lib, workloads

from .conftest import ROOT

torch = pytest.importorskip("torch")
from int4_quantized_moe_amd import device  # noqa: E402

HEADER = open(os.path.join(ROOT, "include", "kt_block.h")).read()
FAKE = 1 << 20  # a non-null, 256-aligned address; never dereferenced by the host checks
NAN, INF = float("nan"), float("inf")


def test_library_exports_every_declared_symbol():
    lib = ctypes.CDLL(_lib.LIBRARY_PATH)
    names = sorted(set(re.findall(r"^(?:int|size_t) (kt_\w+)\(", HEADER, re.M)))
    assert len(names) == 11
    bound = _lib.load_library()
    for name in names:
        assert hasattr(lib, name), name
        assert getattr(bound, name).argtypes is not None, name


def test_constants_match_the_header():
    for name, value in re.findall(r"#define (KT_\w+) (\d+)", HEADER):
        if hasattr(_lib, name):
            assert getattr(_lib, name) == int(value), name
    acts = dict(re.findall(r"#define KT_ACT_(\w+) (\d+)", HEADER))
    assert {k.lower(): int(v) for k, v in acts.items()} == _lib.ACTIVATIONS
    assert _lib.SCORES == {"softmax": 0, "sigmoid": 1} and _lib.CKPT8_FORMATS == {"int8": 0, "e4m3": 1}


def _fails(rc, message, code=kt.KT_RAWINT4_EINVAL):
    assert rc == code, (rc, kt.kt_rawint4_last_error())
    assert message in kt.kt_rawint4_last_error()


# ---------------------------------------------------------------- routing


def _router(**over):
    args = dict(num_experts=64, top_k=4, num_groups=4, top_groups=2, group_top=2, score=0, renormalize=1, scale=1.0,
                logits_type=1)
    args.update(over)
    return kt.kt_router(*args.values())


@pytest.mark.parametrize("over,message", [
    (dict(num_experts=0), "num_experts"), (dict(num_experts=8193), "num_experts"), (dict(top_k=0), "top_k"),
    (dict(top_k=65), "top_k"), (dict(num_groups=0), "num_groups"), (dict(num_groups=3), "num_groups"),
    (dict(num_experts=130, num_groups=65), "num_groups"), (dict(top_groups=0), "top_groups"),
    (dict(top_groups=5), "top_groups"), (dict(group_top=0), "group_top"), (dict(group_top=3), "group_top"),
    (dict(num_groups=64, top_groups=8, group_top=2), "group_top"), (dict(top_k=33), "top_groups groups"),
    (dict(score=2), "score"), (dict(logits_type=2), "logits_type"), (dict(scale=NAN), "scale"), (dict(scale=INF), "scale"),
])
def test_invalid_routers_are_refused(over, message):
    lib, r = _lib.load_library(), _router(**over)
    _fails(lib.kt_router_fwd(ctypes.byref(r), 4, FAKE, None, None, FAKE, FAKE, None, 0, None), message)
    _fails(lib.kt_router_bwd(ctypes.byref(r), 4, FAKE, FAKE, FAKE, FAKE, None), message)


def test_router_arguments_are_refused():
    lib, r = _lib.load_library(), _router()
    fwd = lambda t=4, l=FAKE, b=None, m=None, i=FAKE, w=FAKE, n=None, r=r: lib.kt_router_fwd(  # noqa: E731
        ctypes.byref(r) if r else None, t, l, b, m, i, w, n, 0, None)
    _fails(fwd(r=None), "router is NULL")
    _fails(fwd(t=-1), "tokens")
    _fails(fwd(t=(1 << 23) + 1), "2^23")
    for k in "liw":
        _fails(fwd(**{k: None}), "non-NULL")
    _fails(fwd(l=FAKE + 8), "aligned")
    _fails(fwd(i=FAKE + 4), "aligned")
    _fails(fwd(w=FAKE + 2), "aligned")
    _fails(fwd(b=FAKE + 1), "aligned")
    _fails(fwd(n=FAKE + 2), "aligned")
    bwd = lambda t=4, l=FAKE, i=FAKE, g=FAKE, o=FAKE: lib.kt_router_bwd(ctypes.byref(r), t, l, i, g, o, None)  # noqa: E731
    for k in "ligo":
        _fails(bwd(**{k: None}), "non-NULL")
    _fails(bwd(o=FAKE + 4), "aligned")
    _fails(lib.kt_router_update_bias(FAKE, FAKE, 0, 0.1, None), "num_experts")
    _fails(lib.kt_router_update_bias(None, FAKE, 4, 0.1, None), "non-NULL")
    _fails(lib.kt_router_update_bias(FAKE, FAKE, 4, NAN, None), "rate")
    _fails(lib.kt_router_update_bias(FAKE + 2, FAKE, 4, 0.1, None), "aligned")


def test_router_class_refuses():
    with pytest.raises(ValueError, match="score"):
        device.DeviceRouter(8, 2, score="tanh")
    with pytest.raises(ValueError, match="bias"):
        device.DeviceRouter(8, 2, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="bias"):
        device.DeviceRouter(8, 2, bias=torch.zeros(8, dtype=torch.float64))
    r = device.DeviceRouter(8, 2)
    l = torch.zeros(3, 8)
    for bad, word in ((l.half(), "logits"), (torch.zeros(3, 7), "shape"), (torch.zeros(8), "tokens"),
                      (torch.zeros(8, 3).t(), "contiguous"), (l, "GPU")):
        with pytest.raises(ValueError, match=word):
            r.forward(bad)
    ids, w = torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)
    for kw, word in ((dict(expert_ids=ids.int()), "expert_ids"), (dict(route_weights=w[:2]), "route_weights"),
                     (dict(load=torch.zeros(8)), "load"), (dict(token_mask=torch.zeros(3)), "token_mask"),
                     (dict(token_mask=torch.zeros(4, dtype=torch.bool)), "token_mask"),
                     (dict(expert_ids=torch.zeros(2, 3, dtype=torch.int64).t()), "contiguous")):
        with pytest.raises(ValueError, match=word):
            r.forward(l, **kw)
    for args, word in (((l, ids, w.double()), "grad_route"), ((l, ids[:, :1], w), "expert_ids"),
                       ((l, ids, w, l.bfloat16()), "grad_logits"), ((l, ids, w), "GPU")):
        with pytest.raises(ValueError, match=word):
            r.backward(*args)
    with pytest.raises(ValueError, match="no bias"):
        r.update_bias(torch.zeros(8, dtype=torch.int32), 0.1)


# ---------------------------------------------------------------- checkpoints


def test_checkpoint_arguments_are_refused():
    lib = _lib.load_library()
    for fn in (lambda x, r, c, f, a, b: lib.kt_ckpt8_pack(x, r, c, f, a, b, None),
               lambda x, r, c, f, a, b: lib.kt_ckpt8_unpack(a, b, r, c, f, x, None)):
        _fails(fn(FAKE, -1, 4, 0, FAKE, FAKE), "rows")
        _fails(fn(FAKE, 4, -1, 0, FAKE, FAKE), "rows")
        _fails(fn(FAKE, 1 << 32, 33, 0, FAKE, FAKE), "2^32")
        _fails(fn(FAKE, 2, 1 << 60, 0, FAKE, FAKE), "2^32")
        _fails(fn(FAKE, 4, 4, 2, FAKE, FAKE), "format")
        for args in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
            _fails(fn(args[0], 4, 4, 0, args[1], args[2]), "non-NULL")
        _fails(fn(FAKE + 8, 4, 4, 0, FAKE, FAKE), "aligned")
        _fails(fn(FAKE, 4, 4, 0, FAKE + 2, FAKE), "aligned")
        assert fn(None, 0, 4, 0, None, None) == kt.KT_RAWINT4_OK


def test_checkpoint_class_refuses():
    codes, scales = torch.zeros(3, 40, dtype=torch.int8), torch.zeros(3, 2, dtype=torch.uint8)
    for args, word in (((codes, scales, "int4"), "format"), ((codes.float(), scales, "int8"), "one byte"),
                       ((codes[0], scales, "int8"), "one byte"), ((codes, scales[:, :1], "int8"), "scales"),
                       ((codes, scales.int(), "int8"), "scales"), ((codes.t(), scales, "int8"), "contiguous")):
        with pytest.raises(ValueError, match=word):
            device.Checkpoint8(*args)
    x = torch.zeros(3, 40, dtype=torch.bfloat16)
    out = device.Checkpoint8(codes, scales, "int8")
    for args, word in (((x.float(), "int8", out), "bfloat16"), ((x[0], "int8", out), "rows"), ((x, "e4m3", out), "out"),
                       ((x[:2], "int8", out), "out"), ((x, "int8", out), "GPU"), ((x, "int8"), "GPU")):
        with pytest.raises(ValueError, match=word):
            device.pack_checkpoint8(*args)
    for args, word in (((out, x.float()), "bfloat16"), ((out, x[:2]), "shape"), ((out,), "GPU")):
        with pytest.raises(ValueError, match=word):
            device.unpack_checkpoint8(*args)


def _layer():
    return kt.make_layer(8, 2, 512, 384, 8, 16.0, 2.0, *([FAKE] * 12))


def test_experts_backward_from_a_checkpoint_refuses():
    lib, layer = _lib.load_library(), _layer()
    need = kt.kt_moe_bwd_ckpt8_workspace_bytes(layer, 5)
    assert need == kt.kt_rawint4_moe_workspace_bytes(layer, 5) + 5 * 512 * 2  # a multiple of 256
    with pytest.raises(kt.KtRawInt4Error, match="qlen"):
        kt.kt_moe_bwd_ckpt8_workspace_bytes(layer, -1)

    def call(fmt=0, codes=FAKE, scales=FAKE, ids=FAKE, grads=FAKE, ws=FAKE, nbytes=need, qlen=5):
        return lib.kt_moe_bwd_ckpt8(ctypes.byref(layer), qlen, fmt, codes, scales, ids, FAKE, FAKE, FAKE, None,
                                    *([grads] * 6), 0, 1.0, ws, nbytes, None)

    _fails(call(fmt=2), "format")
    _fails(call(codes=None), "codes")
    _fails(call(scales=None), "codes")
    _fails(call(codes=FAKE + 1), "aligned")
    _fails(call(ids=None), "non-NULL")
    _fails(call(grads=None), "gradient")
    _fails(call(ws=None), "workspace")
    _fails(call(ws=FAKE + 8), "aligned")
    _fails(call(nbytes=need - 256), "smaller", kt.KT_RAWINT4_EWORKSPACE)


def test_layer_class_refuses_a_checkpoint_of_other_sizes():
    layer = object.__new__(device.DeviceLayer)
    layer.cfg = workloads.LayerConfig("small", 8, 2, 64, 32, 4, 8.0, 5, 2.0)
    t = 5
    ck = device.Checkpoint8(torch.zeros(t, 64, dtype=torch.int8), torch.zeros(t, 2, dtype=torch.uint8), "int8")
    narrow = device.Checkpoint8(torch.zeros(t, 32, dtype=torch.int8), torch.zeros(t, 1, dtype=torch.uint8), "int8")
    ids, rw, dy = torch.zeros(t, 2, dtype=torch.int64), torch.zeros(t, 2), torch.zeros(t, 64, dtype=torch.bfloat16)
    for args, kw, word in (((narrow, ids, rw, dy), {}, "checkpoint must be"), ((ck, ids[:4], rw, dy), {}, "expert_ids"),
                           ((ck, ids.int(), rw, dy), {}, "expert_ids"), ((ck, ids, rw[:, :1], dy), {}, "route_weights"),
                           ((ck, ids, rw, dy.float()), {}, "grad_output"), ((ck, ids, rw, dy[:4]), {}, "grad_output"),
                           ((ck, ids, rw, dy), dict(grad_input=dy[:4]), "grad_input"),
                           ((ck, ids, rw, dy), dict(grad_route=rw.double()), "grad_route"),
                           ((ck, ids, rw, dy), {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            layer.backward(*args, None, {}, **kw)


# ---------------------------------------------------------------- dense products


def _linear(k=64, n=24, act=0, weight=FAKE, bias=None):
    return kt.kt_linear(k, n, act, weight, bias)


@pytest.mark.parametrize("over,message", [
    (dict(k=0), "in_features"), (dict(k=12), "in_features"), (dict(k=65544), "in_features"), (dict(n=0), "out_features"),
    (dict(n=65537), "out_features"), (dict(act=-1), "activation"), (dict(act=5), "activation"),
    (dict(weight=None), "weight"), (dict(weight=FAKE + 8), "aligned"), (dict(bias=FAKE + 4), "aligned"),
])
def test_invalid_layers_are_refused(over, message):
    lib, lin = _lib.load_library(), _linear(**over)
    with pytest.raises(kt.KtRawInt4Error, match=message):
        kt.kt_linear_workspace_bytes(lin, 4)
    with pytest.raises(kt.KtRawInt4Error, match=message):
        kt.kt_linear_bwd_workspace_bytes(lin, 4)
    _fails(lib.kt_linear_fwd(ctypes.byref(lin), 4, FAKE, None, FAKE, 0, None, FAKE, 1 << 30, None), message)
    _fails(lib.kt_linear_bwd(ctypes.byref(lin), 4, FAKE, None, None, FAKE, 0, None, FAKE, FAKE, FAKE, 0, 1.0, FAKE,
                             1 << 30, None), message)


def test_linear_arguments_are_refused():
    lib, lin = _lib.load_library(), _linear()

    def fwd(t=200, x=FAKE, r=None, y=FAKE, kind=0, z=None, ws=FAKE, nbytes=1 << 30):
        return lib.kt_linear_fwd(ctypes.byref(lin), t, x, r, y, kind, z, ws, nbytes, None)

    _fails(fwd(t=-1), "tokens")
    _fails(fwd(t=(1 << 20) + 1), "tokens")
    _fails(fwd(x=None), "non-NULL")
    _fails(fwd(y=None), "non-NULL")
    _fails(fwd(kind=2), "output_type")
    for k in "xryz":
        _fails(fwd(**{k: FAKE + 8}), "aligned")
    long = _linear(k=7168)
    need = kt.kt_linear_workspace_bytes(long, 200)
    assert need > 0 and need % 256 == 0
    for ws, nbytes, word, code in ((None, need, "NULL", -1), (FAKE + 8, need, "aligned", -1), (FAKE, need - 1, "smaller", -2)):
        _fails(lib.kt_linear_fwd(ctypes.byref(long), 200, FAKE, None, FAKE, 0, None, ws, nbytes, None), word, code)
    assert kt.kt_linear_workspace_bytes(long, 1) == 0 and kt.kt_linear_workspace_bytes(long, 0) == 0

    act = _linear(act=2)
    ck = kt.kt_ckpt8(0, FAKE, FAKE)

    def bwd(lin=lin, t=200, x=FAKE, ck=None, z=None, dy=FAKE, kind=0, r=None, dx=FAKE, dw=FAKE, db=None, scale=1.0,
            ws=FAKE, nbytes=1 << 40):
        return lib.kt_linear_bwd(ctypes.byref(lin), t, x, None if ck is None else ctypes.byref(ck), z, dy, kind, r, dx,
                                 dw, db, 0, scale, ws, nbytes, None)

    _fails(bwd(kind=3), "grad_output_type")
    _fails(bwd(scale=INF), "grad_scale")
    _fails(bwd(ck=ck), "not both")
    _fails(bwd(x=None, ck=kt.kt_ckpt8(3, FAKE, FAKE)), "format")
    _fails(bwd(x=None), "inputs")
    _fails(bwd(x=None, ck=kt.kt_ckpt8(0, FAKE, None)), "inputs")
    _fails(bwd(x=None, ck=kt.kt_ckpt8(0, FAKE + 2, FAKE)), "aligned")
    _fails(bwd(dy=None), "grad_output")
    _fails(bwd(lin=act), "preact")
    for k in ("x", "dy", "r", "dx", "dw", "db"):
        _fails(bwd(**{k: FAKE + 8}), "aligned")
    need = kt.kt_linear_bwd_workspace_bytes(lin, 200)
    assert kt.kt_linear_bwd_workspace_bytes(lin, 200, True) == need + 200 * 64 * 2
    _fails(bwd(nbytes=need - 1), "smaller", kt.KT_RAWINT4_EWORKSPACE)
    _fails(bwd(x=None, ck=ck, nbytes=need), "smaller", kt.KT_RAWINT4_EWORKSPACE)
    _fails(bwd(ws=None), "NULL")


def test_workspace_plans_over_the_range():
    for k in (8, 64, 2048, 65536):
        for n in (1, 7, 384, 65536):
            last = 0
            for t in (0, 1, 17, 128, 4096, 1 << 20):
                lin = _linear(k=k, n=n)
                fwd, bwd = kt.kt_linear_workspace_bytes(lin, t), kt.kt_linear_bwd_workspace_bytes(lin, t, True)
                assert fwd % 256 == 0 and bwd % 256 == 0 and bwd >= 0
                # three planes of dz, the unpacked rows, a bounded number of partial sums
                outputs = max(t * k, n * k, t * n)
                assert bwd <= 6 * t * (n + 8) + 2 * t * k + 4 * n * (t // 32 + 2) + 4 * 65 * outputs + 4096
                last = max(last, bwd)


def test_linear_class_refuses():
    w = torch.zeros(24, 64, dtype=torch.bfloat16)
    for args, word in (((w.float(),), "bfloat16"), ((w[0],), "weight"), ((w.t(),), "contiguous"),
                       ((w, torch.zeros(23)), "bias"), ((w, torch.zeros(24).bfloat16()), "bias"),
                       ((w, None, "swish"), "activation")):
        with pytest.raises(ValueError, match=word):
            device.DeviceLinear(*args)
    lin = device.DeviceLinear(w, torch.zeros(24), "silu")
    x, y = torch.zeros(5, 64, dtype=torch.bfloat16), torch.zeros(5, 24, dtype=torch.bfloat16)
    for args, kw, word in (((x.float(), None), {}, "bfloat16"), ((x[:, :32], None), {}, "shape"), ((x[0], None), {}, "x must"),
                           ((x, None), dict(residual=y[:4]), "residual"), ((x, None), dict(preact=y.float()), "preact"),
                           ((x, None), dict(output=y.half()), "output"), ((x, None), dict(output=y[:, :8]), "output"),
                           ((x, None), dict(dtype=torch.float16), "output"), ((x, None), {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            lin.forward(*args, **kw)
    g = {"weight": torch.zeros(24, 64), "bias": torch.zeros(24)}
    ck = device.Checkpoint8(torch.zeros(5, 32, dtype=torch.int8), torch.zeros(5, 1, dtype=torch.uint8), "int8")
    for args, kw, word in (((x, y.double(), None, g), {}, "grad_output"), ((x, y[:4], None, g), {}, "grad_output"),
                           ((ck, y, None, g), {}, "tokens"), ((x, y, None, {"weight": w}), {}, "weight"),
                           ((x, y, None, {"bias": torch.zeros(3)}), {}, "bias"),
                           ((x, y, None, g), dict(preact=y[:3]), "preact"),
                           ((x, y, None, g), dict(grad_input=x.float()), "grad_input"),
                           ((x, y, None, g), dict(grad_residual=x[:1]), "grad_residual"), ((x, y, None, g), {}, "GPU")):
        with pytest.raises(ValueError, match=word):
            lin.backward(*args, **kw)


# ---------------------------------------------------------------- plain C


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_plain_c_consumer(tmp_path):
    lib_dir = os.path.dirname(_lib.LIBRARY_PATH)
    exe = tmp_path / "block_consumer"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "block_consumer.c"), "-o", str(exe), "-L", lib_dir,
                    "-l:libkt_rawint4.so", f"-Wl,-rpath,{lib_dir}", "-lm"], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "FAIL" not in run.stdout and run.stdout.count("ok   ") == 17
