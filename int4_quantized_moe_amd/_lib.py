"""ctypes binding of ``libkt_rawint4.so`` (argument marshalling only).

Every function has the name and argument order of its C entry point in
``include/kt_rawint4.h`` or ``include/kt_block.h``.  Tensors are passed as raw pointers (``data_ptr()``),
``stream`` defaults to torch's current HIP stream, and a nonzero return code
raises ``KtRawInt4Error`` with the library's message.  There is no fallback:
without the built library every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libkt_rawint4.so")

KT_RAWINT4_OK = 0
KT_RAWINT4_EINVAL = -1
KT_RAWINT4_EWORKSPACE = -2
KT_RAWINT4_EHIP = -3

KT_RAWINT4_STATIC_SCRATCH_BYTES = 64 << 20

KT_RAWINT4_FORMAT_RAWINT4 = 0
KT_RAWINT4_FORMAT_MXFP4 = 1
FORMATS = {"rawint4": KT_RAWINT4_FORMAT_RAWINT4, "mxfp4": KT_RAWINT4_FORMAT_MXFP4}

KT_TYPE_BF16 = 0
KT_TYPE_F32 = 1
KT_SCORE_SOFTMAX = 0
KT_SCORE_SIGMOID = 1
SCORES = {"softmax": KT_SCORE_SOFTMAX, "sigmoid": KT_SCORE_SIGMOID}
KT_ROUTER_MAX_GROUPS = 64
KT_CKPT8_INT8 = 0
KT_CKPT8_E4M3 = 1
CKPT8_FORMATS = {"int8": KT_CKPT8_INT8, "e4m3": KT_CKPT8_E4M3}
KT_CKPT8_GROUP = 32
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_vp = ctypes.c_void_p


class KtRawInt4Error(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"kt_rawint4 error {code}: {message}")
        self.code = code


class kt_rawint4_moe_layer(ctypes.Structure):  # noqa: N801 - the C struct's name
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("intermediate", ctypes.c_int32),
        ("rank", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("swiglu_limit", ctypes.c_float),
        ("gate_packed", _vp),
        ("up_packed", _vp),
        ("down_packed", _vp),
        ("gate_scale", _vp),
        ("up_scale", _vp),
        ("down_scale", _vp),
        ("gate_lora_a", _vp),
        ("gate_lora_b", _vp),
        ("up_lora_a", _vp),
        ("up_lora_b", _vp),
        ("down_lora_a", _vp),
        ("down_lora_b", _vp),
        ("weight_format", ctypes.c_int32),
    ]


class kt_router(ctypes.Structure):  # noqa: N801 - the C struct's name
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_top", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("logits_type", ctypes.c_int32),
    ]


class kt_linear(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("weight", _vp),
        ("bias", _vp),
    ]


class kt_ckpt8(ctypes.Structure):  # noqa: N801
    _fields_ = [("format", ctypes.c_int32), ("codes", _vp), ("scales", _vp)]


_lib = None


def load_library() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise KtRawInt4Error(KT_RAWINT4_EHIP, f"{LIBRARY_PATH} is not built; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIBRARY_PATH)
    lp = ctypes.POINTER(kt_rawint4_moe_layer)
    rp, np_, cp = ctypes.POINTER(kt_router), ctypes.POINTER(kt_linear), ctypes.POINTER(kt_ckpt8)
    i32, i64, f32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sigs = {
        "kt_rawint4_moe_workspace_bytes": (sz, [lp, i32]),
        "kt_rawint4_moe_fwd": (ctypes.c_int, [lp, i32, _vp, _vp, _vp, _vp, _vp, sz, _vp]),
        "kt_rawint4_moe_infer_workspace_bytes": (sz, [lp, i32]),
        "kt_rawint4_moe_infer": (ctypes.c_int, [lp, i32, _vp, _vp, _vp, _vp, _vp, sz, _vp]),
        "kt_rawint4_moe_infer_static": (ctypes.c_int, [lp, i32, _vp, _vp, _vp, _vp, _vp]),
        "kt_rawint4_moe_bwd": (ctypes.c_int, [lp, i32, _vp, _vp, _vp, _vp, _vp, _vp] + [_vp] * 6 + [i32, f32, _vp, sz, _vp]),
        "kt_rawint4_moe_bwd_recompute": (ctypes.c_int,
                                         [lp, i32, _vp, _vp, _vp, _vp, _vp, _vp] + [_vp] * 6 + [i32, f32, _vp, sz, _vp]),
        "kt_moe_bwd_ckpt8_workspace_bytes": (sz, [lp, i32]),
        "kt_moe_bwd_ckpt8": (ctypes.c_int,
                             [lp, i32, i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp] + [_vp] * 6 + [i32, f32, _vp, sz, _vp]),
        "kt_ckpt8_pack": (ctypes.c_int, [_vp, i64, i64, i32, _vp, _vp, _vp]),
        "kt_ckpt8_unpack": (ctypes.c_int, [_vp, _vp, i64, i64, i32, _vp, _vp]),
        "kt_router_fwd": (ctypes.c_int, [rp, i32, _vp, _vp, _vp, _vp, _vp, _vp, i32, _vp]),
        "kt_router_bwd": (ctypes.c_int, [rp, i32, _vp, _vp, _vp, _vp, _vp]),
        "kt_router_update_bias": (ctypes.c_int, [_vp, _vp, i32, f32, _vp]),
        "kt_linear_workspace_bytes": (sz, [np_, i32]),
        "kt_linear_fwd": (ctypes.c_int, [np_, i32, _vp, _vp, _vp, i32, _vp, _vp, sz, _vp]),
        "kt_linear_bwd_workspace_bytes": (sz, [np_, i32, i32]),
        "kt_linear_bwd": (ctypes.c_int,
                          [np_, i32, _vp, cp, _vp, _vp, i32, _vp, _vp, _vp, _vp, i32, f32, _vp, sz, _vp]),
        "kt_rawint4_unpack": (ctypes.c_int, [_vp, i64, i64, _vp, _vp]),
        "kt_rawint4_dequant": (ctypes.c_int, [_vp, _vp, i64, i64, _vp, _vp]),
        "kt_rawint4_dequant_mxfp4": (ctypes.c_int, [_vp, _vp, i64, i64, _vp, _vp]),
        "kt_rawint4_group_workspace_bytes": (sz, [i32, i32, i32]),
        "kt_rawint4_group": (ctypes.c_int, [_vp, i32, i32, i32, _vp, _vp, _vp, sz, _vp]),
        "kt_rawint4_moe_diagnostics": (ctypes.c_int, [_vp, sz, ctypes.POINTER(i64), ctypes.POINTER(i64), _vp]),
        "kt_rawint4_moe_saved_preactivations": (ctypes.c_int, [lp, i32, _vp, sz, _vp, _vp, _vp]),
        "kt_rawint4_profile_enable": (ctypes.c_int, [i32]),
        "kt_rawint4_profile_read": (ctypes.c_int, [_vp, _vp, i32]),
        "kt_rawint4_profile_phase_name": (ctypes.c_char_p, [i32]),
        "kt_rawint4_last_error": (ctypes.c_char_p, []),
        "kt_rawint4_weight_layout": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to kt_rawint4 must be contiguous")
    return t.data_ptr()


_raw_stream = None


def device_stream(index: int) -> int:
    """The handle of torch's current stream on GPU ``index``."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        # 0.1 us; a Stream object takes 2.5
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(index)


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch

        return device_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int) -> None:
    if rc != KT_RAWINT4_OK:
        raise KtRawInt4Error(rc, kt_rawint4_last_error())


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def make_layer(num_experts, top_k, hidden, intermediate, rank, alpha, swiglu_limit, gate_packed, up_packed,
               down_packed, gate_scale, up_scale, down_scale, gate_lora_a, gate_lora_b, up_lora_a, up_lora_b,
               down_lora_a, down_lora_b, weight_format=KT_RAWINT4_FORMAT_RAWINT4) -> kt_rawint4_moe_layer:
    """Fill the C layer struct; the caller keeps the tensors alive.  weight_format:
    KT_RAWINT4_FORMAT_* or its name ("rawint4", "mxfp4")."""
    fmt = FORMATS[weight_format] if isinstance(weight_format, str) else int(weight_format)
    return kt_rawint4_moe_layer(int(num_experts), int(top_k), int(hidden), int(intermediate), int(rank), float(alpha),
                                float(swiglu_limit), _ptr(gate_packed), _ptr(up_packed), _ptr(down_packed),
                                _ptr(gate_scale), _ptr(up_scale), _ptr(down_scale), _ptr(gate_lora_a),
                                _ptr(gate_lora_b), _ptr(up_lora_a), _ptr(up_lora_b), _ptr(down_lora_a),
                                _ptr(down_lora_b), fmt)


def kt_rawint4_moe_workspace_bytes(layer: kt_rawint4_moe_layer, qlen: int) -> int:
    n = load_library().kt_rawint4_moe_workspace_bytes(ctypes.byref(layer), int(qlen))
    if n == 0:
        raise KtRawInt4Error(KT_RAWINT4_EINVAL, kt_rawint4_last_error())
    return int(n)


def kt_rawint4_moe_fwd(layer, qlen, inputs, expert_ids, route_weights, output, workspace, stream=None) -> None:
    _check(load_library().kt_rawint4_moe_fwd(ctypes.byref(layer), int(qlen), _ptr(inputs), _ptr(expert_ids),
                                             _ptr(route_weights), _ptr(output), _ptr(workspace),
                                             _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_rawint4_moe_infer_workspace_bytes(layer: kt_rawint4_moe_layer, qlen: int) -> int:
    n = load_library().kt_rawint4_moe_infer_workspace_bytes(ctypes.byref(layer), int(qlen))
    if n == 0:
        raise KtRawInt4Error(KT_RAWINT4_EINVAL, kt_rawint4_last_error())
    return int(n)


def kt_rawint4_moe_infer(layer, qlen, inputs, expert_ids, route_weights, output, workspace, stream=None) -> None:
    _check(load_library().kt_rawint4_moe_infer(ctypes.byref(layer), int(qlen), _ptr(inputs), _ptr(expert_ids),
                                               _ptr(route_weights), _ptr(output), _ptr(workspace),
                                               _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_rawint4_moe_infer_static(layer, qlen, inputs, expert_ids, route_weights, output, stream=None) -> None:
    _check(load_library().kt_rawint4_moe_infer_static(ctypes.byref(layer), int(qlen), _ptr(inputs), _ptr(expert_ids),
                                                      _ptr(route_weights), _ptr(output), _stream(stream)))


def kt_rawint4_moe_bwd(layer, qlen, inputs, expert_ids, route_weights, grad_output, grad_input, grad_route, d_gate_a,
                       d_gate_b, d_up_a, d_up_b, d_down_a, d_down_b, accumulate, grad_scale, workspace,
                       stream=None) -> None:
    _check(load_library().kt_rawint4_moe_bwd(
        ctypes.byref(layer), int(qlen), _ptr(inputs), _ptr(expert_ids), _ptr(route_weights), _ptr(grad_output),
        _ptr(grad_input), _ptr(grad_route), _ptr(d_gate_a), _ptr(d_gate_b), _ptr(d_up_a), _ptr(d_up_b),
        _ptr(d_down_a), _ptr(d_down_b), int(bool(accumulate)), float(grad_scale), _ptr(workspace),
        _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_rawint4_moe_bwd_recompute(layer, qlen, inputs, expert_ids, route_weights, grad_output, grad_input, grad_route,
                                 d_gate_a, d_gate_b, d_up_a, d_up_b, d_down_a, d_down_b, accumulate, grad_scale,
                                 workspace, stream=None) -> None:
    _check(load_library().kt_rawint4_moe_bwd_recompute(
        ctypes.byref(layer), int(qlen), _ptr(inputs), _ptr(expert_ids), _ptr(route_weights), _ptr(grad_output),
        _ptr(grad_input), _ptr(grad_route), _ptr(d_gate_a), _ptr(d_gate_b), _ptr(d_up_a), _ptr(d_up_b),
        _ptr(d_down_a), _ptr(d_down_b), int(bool(accumulate)), float(grad_scale), _ptr(workspace),
        _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_moe_bwd_ckpt8_workspace_bytes(layer: kt_rawint4_moe_layer, qlen: int) -> int:
    n = load_library().kt_moe_bwd_ckpt8_workspace_bytes(ctypes.byref(layer), int(qlen))
    if n == 0:
        raise KtRawInt4Error(KT_RAWINT4_EINVAL, kt_rawint4_last_error())
    return int(n)


def kt_moe_bwd_ckpt8(layer, qlen, format, codes, scales, expert_ids, route_weights, grad_output, grad_input, grad_route,
                     d_gate_a, d_gate_b, d_up_a, d_up_b, d_down_a, d_down_b, accumulate, grad_scale, workspace,
                     stream=None) -> None:
    _check(load_library().kt_moe_bwd_ckpt8(
        ctypes.byref(layer), int(qlen), int(format), _ptr(codes), _ptr(scales), _ptr(expert_ids), _ptr(route_weights),
        _ptr(grad_output), _ptr(grad_input), _ptr(grad_route), _ptr(d_gate_a), _ptr(d_gate_b), _ptr(d_up_a),
        _ptr(d_up_b), _ptr(d_down_a), _ptr(d_down_b), int(bool(accumulate)), float(grad_scale), _ptr(workspace),
        _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_ckpt8_pack(x, rows, cols, format, codes, scales, stream=None) -> None:
    _check(load_library().kt_ckpt8_pack(_ptr(x), rows, cols, format, _ptr(codes), _ptr(scales), _stream(stream)))


def kt_ckpt8_unpack(codes, scales, rows, cols, format, x, stream=None) -> None:
    _check(load_library().kt_ckpt8_unpack(_ptr(codes), _ptr(scales), rows, cols, format, _ptr(x), _stream(stream)))


def kt_router_fwd(router, tokens, logits, bias, token_mask, expert_ids, route_weights, load, accumulate,
                  stream=None) -> None:
    _check(load_library().kt_router_fwd(ctypes.byref(router), tokens, _ptr(logits), _ptr(bias), _ptr(token_mask),
                                        _ptr(expert_ids), _ptr(route_weights), _ptr(load), int(bool(accumulate)),
                                        _stream(stream)))


def kt_router_bwd(router, tokens, logits, expert_ids, grad_route, grad_logits, stream=None) -> None:
    _check(load_library().kt_router_bwd(ctypes.byref(router), tokens, _ptr(logits), _ptr(expert_ids),
                                        _ptr(grad_route), _ptr(grad_logits), _stream(stream)))


def kt_router_update_bias(bias, load, num_experts, rate, stream=None) -> None:
    _check(load_library().kt_router_update_bias(_ptr(bias), _ptr(load), int(num_experts), float(rate),
                                                _stream(stream)))


def make_linear(weight, bias=None, activation="none") -> kt_linear:
    """Fill the C struct of a dense layer from its weight [out, in]; the caller keeps the tensors alive."""
    return kt_linear(int(weight.shape[1]), int(weight.shape[0]), ACTIVATIONS[activation], _ptr(weight), _ptr(bias))


def _checked_size(n: int) -> int:
    # a size of 0 is a valid answer; an error leaves its message
    if n == 0 and kt_rawint4_last_error():
        raise KtRawInt4Error(KT_RAWINT4_EINVAL, kt_rawint4_last_error())
    return int(n)


def kt_linear_workspace_bytes(linear, tokens) -> int:
    return _checked_size(load_library().kt_linear_workspace_bytes(ctypes.byref(linear), int(tokens)))


def kt_linear_fwd(linear, tokens, inputs, residual, output, output_type, preact, workspace, stream=None) -> None:
    _check(load_library().kt_linear_fwd(ctypes.byref(linear), tokens, _ptr(inputs), _ptr(residual), _ptr(output),
                                        output_type, _ptr(preact), _ptr(workspace),
                                        _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_linear_bwd_workspace_bytes(linear, tokens, from_checkpoint=False) -> int:
    return _checked_size(load_library().kt_linear_bwd_workspace_bytes(ctypes.byref(linear), int(tokens),
                                                                      int(bool(from_checkpoint))))


def kt_linear_bwd(linear, tokens, inputs, checkpoint, preact, grad_output, grad_output_type, grad_residual, grad_input,
                  d_weight, d_bias, accumulate, grad_scale, workspace, stream=None) -> None:
    _check(load_library().kt_linear_bwd(
        ctypes.byref(linear), tokens, _ptr(inputs), None if checkpoint is None else ctypes.byref(checkpoint),
        _ptr(preact), _ptr(grad_output), grad_output_type, _ptr(grad_residual), _ptr(grad_input), _ptr(d_weight),
        _ptr(d_bias), int(bool(accumulate)), float(grad_scale), _ptr(workspace),
        _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_rawint4_unpack(packed, n, k, codes, stream=None) -> None:
    _check(load_library().kt_rawint4_unpack(_ptr(packed), int(n), int(k), _ptr(codes), _stream(stream)))


def kt_rawint4_dequant(packed, scales, n, k, weights, stream=None) -> None:
    _check(load_library().kt_rawint4_dequant(_ptr(packed), _ptr(scales), int(n), int(k), _ptr(weights),
                                             _stream(stream)))


def kt_rawint4_dequant_mxfp4(packed, scales, n, k, weights, stream=None) -> None:
    _check(load_library().kt_rawint4_dequant_mxfp4(_ptr(packed), _ptr(scales), int(n), int(k), _ptr(weights),
                                                   _stream(stream)))


def kt_rawint4_group_workspace_bytes(qlen, top_k, num_experts) -> int:
    n = load_library().kt_rawint4_group_workspace_bytes(int(qlen), int(top_k), int(num_experts))
    if n == 0:
        raise KtRawInt4Error(KT_RAWINT4_EINVAL, kt_rawint4_last_error())
    return int(n)


def kt_rawint4_group(expert_ids, qlen, top_k, num_experts, offsets, sorted_slot, workspace, stream=None) -> None:
    _check(load_library().kt_rawint4_group(_ptr(expert_ids), int(qlen), int(top_k), int(num_experts), _ptr(offsets),
                                           _ptr(sorted_slot), _ptr(workspace),
                                           _nbytes(workspace) if workspace is not None else 0, _stream(stream)))


def kt_rawint4_moe_diagnostics(workspace, stream=None):
    """Returns (bad_ids, bad_scales) of the latest forward; synchronises the stream."""
    a, b = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(load_library().kt_rawint4_moe_diagnostics(_ptr(workspace), _nbytes(workspace), ctypes.byref(a),
                                                     ctypes.byref(b), _stream(stream)))
    return int(a.value), int(b.value)


def kt_rawint4_moe_saved_preactivations(layer, qlen, workspace, gate, up, stream=None) -> None:
    _check(load_library().kt_rawint4_moe_saved_preactivations(ctypes.byref(layer), int(qlen), _ptr(workspace),
                                                              _nbytes(workspace), _ptr(gate), _ptr(up),
                                                              _stream(stream)))


def kt_rawint4_profile_enable(on: bool) -> None:
    _check(load_library().kt_rawint4_profile_enable(1 if on else 0))


def kt_rawint4_profile_read():
    """{phase name: (milliseconds, launches)} recorded since the last read."""
    cap = 64
    ms = (ctypes.c_float * cap)()
    n = (ctypes.c_int32 * cap)()
    rc = load_library().kt_rawint4_profile_read(ctypes.addressof(ms), ctypes.addressof(n), cap)
    if rc < 0:
        raise KtRawInt4Error(rc, kt_rawint4_last_error())
    return {kt_rawint4_profile_phase_name(i): (float(ms[i]), int(n[i])) for i in range(rc)}


def kt_rawint4_profile_phase_name(phase: int) -> str:
    return load_library().kt_rawint4_profile_phase_name(int(phase)).decode()


def kt_rawint4_last_error() -> str:
    return load_library().kt_rawint4_last_error().decode()


def kt_rawint4_weight_layout() -> str:
    return load_library().kt_rawint4_weight_layout().decode()
