"""Device-resident layer: uploads a workload to HIP memory and calls the C ABI.

Only allocation and marshalling happen here (torch is used for device memory
and streams); every step of the computation runs in ``libkt_rawint4.so``.
"""

from __future__ import annotations

from typing import Dict, Optional

import numpy as np
import torch

from . import _lib
from .workloads import LORA_NAMES, LayerConfig, Weights


def bf16_tensor(bits: np.ndarray, device) -> torch.Tensor:
    """uint16 bf16 bit patterns (numpy) -> torch.bfloat16 tensor on ``device``."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(torch.bfloat16)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class DeviceLayer:
    """One MoE layer in device memory.  ``base_only=True`` uploads no LoRA and
    passes NULL for all six LoRA pointers: such a layer serves only the
    inference forward of the frozen base."""

    def __init__(self, cfg: LayerConfig, weights: Weights, device="cuda", lora: Optional[Dict[str, np.ndarray]] = None,
                 base_only: bool = False):
        self.cfg = cfg
        self.device = torch.device(device)
        dev = self.device
        self.gate_packed = torch.from_numpy(weights.gate_packed).to(dev)
        self.up_packed = torch.from_numpy(weights.up_packed).to(dev)
        self.down_packed = torch.from_numpy(weights.down_packed).to(dev)
        self.gate_scale = bf16_tensor(weights.gate_scale, dev)
        self.up_scale = bf16_tensor(weights.up_scale, dev)
        self.down_scale = bf16_tensor(weights.down_scale, dev)
        if base_only:
            self.lora = {n: None for n in LORA_NAMES}
        else:
            src = weights.lora if lora is None else lora
            self.lora = {n: torch.from_numpy(np.ascontiguousarray(src[n], dtype=np.float32)).to(dev)
                         for n in LORA_NAMES}
        self.layer = _lib.make_layer(cfg.num_experts, cfg.top_k, cfg.hidden, cfg.intermediate, cfg.rank, cfg.alpha,
                                     cfg.swiglu_limit, self.gate_packed, self.up_packed, self.down_packed,
                                     self.gate_scale, self.up_scale, self.down_scale,
                                     *(self.lora[n] for n in LORA_NAMES), weight_format=cfg.weight_format)

    @classmethod
    def from_tensors(cls, cfg: LayerConfig, weights: Dict[str, torch.Tensor],
                     lora: Optional[Dict[str, torch.Tensor]] = None) -> "DeviceLayer":
        """A layer on tensors that are on the GPU already, used as they are: ``weights`` has gate_packed,
        up_packed and down_packed [E, N, K/2] uint8 and gate_scale, up_scale and down_scale [E, N, K/32]
        bf16; ``lora`` the six LoRA tensors (fp32), or None for the frozen base alone."""
        dev = weights["gate_packed"].device
        e, h, i = cfg.num_experts, cfg.hidden, cfg.intermediate
        self = cls.__new__(cls)
        self.cfg, self.device = cfg, dev
        for name, n, k in (("gate", i, h), ("up", i, h), ("down", h, i)):
            _checked(name + "_packed", weights[name + "_packed"], (e, n, k // 2), torch.uint8, dev)
            _checked(name + "_scale", weights[name + "_scale"], (e, n, k // 32), torch.bfloat16, dev)
            setattr(self, name + "_packed", weights[name + "_packed"])
            setattr(self, name + "_scale", weights[name + "_scale"])
        if lora is not None:
            for name, shape in cfg.lora_shapes().items():
                if lora.get(name) is None:
                    raise ValueError(f"lora has no {name!r}")
                _checked(name, lora[name], shape, torch.float32, dev)
        self.lora = {n: None if lora is None else lora[n] for n in LORA_NAMES}
        self.layer = _lib.make_layer(cfg.num_experts, cfg.top_k, h, i, cfg.rank, cfg.alpha, cfg.swiglu_limit,
                                     self.gate_packed, self.up_packed, self.down_packed, self.gate_scale,
                                     self.up_scale, self.down_scale, *(self.lora[n] for n in LORA_NAMES),
                                     weight_format=cfg.weight_format)
        return self

    def workspace(self, qlen: int) -> torch.Tensor:
        n = _lib.kt_rawint4_moe_workspace_bytes(self.layer, qlen)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def infer_workspace(self, qlen: int) -> torch.Tensor:
        n = _lib.kt_rawint4_moe_infer_workspace_bytes(self.layer, qlen)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def decode_workspace(self, tokens: int) -> torch.Tensor:
        """Of decode() for up to so many tokens."""
        n = _lib.kt_moe_decode_workspace_bytes(self.layer, tokens)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def checkpoint_workspace(self, qlen: int) -> torch.Tensor:
        """Workspace of a backward whose inputs are a Checkpoint8, for that qlen."""
        n = _lib.kt_moe_bwd_ckpt8_workspace_bytes(self.layer, qlen)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def grad_buffers(self, fill: Optional[float] = None) -> Dict[str, torch.Tensor]:
        shapes = self.cfg.lora_shapes()
        if fill is None:
            return {n: torch.empty(shapes[n], dtype=torch.float32, device=self.device) for n in LORA_NAMES}
        return {n: torch.full(shapes[n], fill, dtype=torch.float32, device=self.device) for n in LORA_NAMES}

    def forward(self, inputs, expert_ids, route_weights, workspace, output=None, stream=None) -> torch.Tensor:
        qlen = inputs.shape[0]
        if output is None:
            output = torch.empty((qlen, self.cfg.hidden), dtype=torch.bfloat16, device=self.device)
        _lib.kt_rawint4_moe_fwd(self.layer, qlen, inputs, expert_ids, route_weights, output, workspace, stream)
        return output

    def infer(self, inputs, expert_ids, route_weights, workspace, output=None, stream=None) -> torch.Tensor:
        """Forward that keeps nothing for a backward (the output equals forward()'s)."""
        qlen = inputs.shape[0]
        if output is None:
            output = torch.empty((qlen, self.cfg.hidden), dtype=torch.bfloat16, device=self.device)
        _lib.kt_rawint4_moe_infer(self.layer, qlen, inputs, expert_ids, route_weights, output, workspace, stream)
        return output

    def decode(self, inputs, expert_ids, route_weights, workspace, output=None, stream=None) -> torch.Tensor:
        """infer() for a few tokens (at most KT_MOE_DECODE_MAX_TOKENS, and KT_MOE_DECODE_MAX_SLOTS
        token-slots; hidden at most KT_MOE_DECODE_MAX_HIDDEN), in a decode_workspace().  As measured
        the faster of the two while the experts in use have up to about 2 token-slots each on average (about 6 where
        8 experts are in use); for tokens that share experts more infer() is, by up to 6 times."""
        dev, h, k = self.gate_packed.device, self.cfg.hidden, self.cfg.top_k
        if inputs.dim() != 2:
            raise ValueError("inputs must be [tokens, hidden]")
        tokens = inputs.shape[0]
        _checked("inputs", inputs, (tokens, h), torch.bfloat16, dev)
        _checked("expert_ids", expert_ids, (tokens, k), torch.int64, dev)
        _checked("route_weights", route_weights, (tokens, k), torch.float32, dev)
        _checked("output", output, (tokens, h), torch.bfloat16, dev)
        if _elsewhere(_gpu(inputs)):
            with torch.cuda.device(dev):
                return self.decode(inputs, expert_ids, route_weights, workspace, output, stream)
        _workspace(workspace, dev)
        if output is None:
            output = _empty((tokens, h), torch.bfloat16, dev, stream)
        _lib.kt_moe_decode(self.layer, tokens, inputs, expert_ids, route_weights, output, workspace,
                           _handle(stream, dev))
        return output

    def backward(self, inputs, expert_ids, route_weights, grad_output, workspace, grads, accumulate=False,
                 grad_scale=1.0, grad_input=None, grad_route=None, stream=None, recompute=False):
        """recompute=True: the workspace need not hold this call's forward (it is rerun first).
        ``inputs`` may be a Checkpoint8 of the forward's inputs: the backward then always reruns the
        forward, in a checkpoint_workspace()."""
        qlen = inputs.shape[0]
        if isinstance(inputs, Checkpoint8):
            dev, rows, slots = inputs.codes.device, (qlen, self.cfg.hidden), (qlen, self.cfg.top_k)
            if inputs.shape != rows:
                raise ValueError(f"the checkpoint must be [tokens, {self.cfg.hidden}], not {inputs.shape}")
            for name, t, shape, dtype in (
                    ("expert_ids", expert_ids, slots, torch.int64), ("route_weights", route_weights, slots, torch.float32),
                    ("grad_output", grad_output, rows, torch.bfloat16), ("grad_input", grad_input, rows, torch.bfloat16),
                    ("grad_route", grad_route, slots, torch.float32)):
                _checked(name, t, shape, dtype, dev)
            _workspace(workspace, _gpu(inputs.codes))
            if dev != self.gate_packed.device:
                raise ValueError(f"the checkpoint must be on {self.gate_packed.device}, not on {dev}")
            for name, shape in self.cfg.lora_shapes().items():
                if grads.get(name) is None:
                    raise ValueError(f"grads has no {name!r}")
                _checked(f"grads[{name!r}]", grads[name], shape, torch.float32, dev)
            if _elsewhere(dev):
                with torch.cuda.device(dev):
                    return self.backward(inputs, expert_ids, route_weights, grad_output, workspace, grads, accumulate,
                                         grad_scale, grad_input, grad_route, stream)
            if grad_input is None:
                grad_input = _empty(rows, torch.bfloat16, dev, stream)
            _lib.kt_moe_bwd_ckpt8(self.layer, qlen, inputs.fmt, inputs.codes, inputs.scales, expert_ids, route_weights,
                                  grad_output, grad_input, grad_route, *(grads[n] for n in LORA_NAMES), accumulate,
                                  grad_scale, workspace, stream)
            return grad_input, grad_route
        if grad_input is None:
            grad_input = torch.empty((qlen, self.cfg.hidden), dtype=torch.bfloat16, device=self.device)
        fn = _lib.kt_rawint4_moe_bwd_recompute if recompute else _lib.kt_rawint4_moe_bwd
        fn(self.layer, qlen, inputs, expert_ids, route_weights, grad_output, grad_input, grad_route,
           *(grads[n] for n in LORA_NAMES), accumulate, grad_scale, workspace, stream)
        return grad_input, grad_route

    def saved_preactivations(self, qlen, workspace, stream=None):
        """Gate and up pre-activations of the latest forward in ``workspace``, [qlen, k, I] fp32 each."""
        shape = (qlen, self.cfg.top_k, self.cfg.intermediate)
        gate = torch.empty(shape, dtype=torch.float32, device=self.device)
        up = torch.empty(shape, dtype=torch.float32, device=self.device)
        _lib.kt_rawint4_moe_saved_preactivations(self.layer, qlen, workspace, gate, up, stream)
        return gate, up


class DeviceBatch:
    def __init__(self, batch, device="cuda"):
        dev = torch.device(device)
        self.inputs = bf16_tensor(batch.inputs, dev)
        self.expert_ids = torch.from_numpy(np.ascontiguousarray(batch.expert_ids, dtype=np.int64)).to(dev)
        self.route_weights = torch.from_numpy(np.ascontiguousarray(batch.route_weights, dtype=np.float32)).to(dev)
        self.grad_output = bf16_tensor(batch.grad_output, dev)
        self.qlen = self.inputs.shape[0]


# ---------------------------------------------------------------- operators around the experts


def _checked(name, t, shape, dtype, device):
    """The argument check of every tensor below: type, shape, density and device."""
    if t is None:
        return
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, not {t.device}")


def _gpu(t):
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a GPU, not on {t.device}")
    return t.device


def _stream_object(stream, device):
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=device)
    return stream


def _empty(shape, dtype, device, stream):
    """An output made by a call: it belongs to the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


# (current_device() asks first whether the GPUs are in use; a tensor on one answers that)
_current_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(device) -> bool:
    """Whether another GPU than the tensors' is the current one (a call then makes theirs current for its time)."""
    return _current_index() != device.index


def _handle(stream, device):
    """``stream``, or the device's current one."""
    return _lib.device_stream(device.index) if stream is None else stream


def _workspace(workspace, device) -> None:
    if workspace is not None and workspace.device != device:
        raise ValueError(f"the workspace must be on {device}, not on {workspace.device}")


_TYPES = {torch.bfloat16: _lib.KT_TYPE_BF16, torch.float32: _lib.KT_TYPE_F32}


class Checkpoint8:
    """Rows of bf16 kept in 8 bits: ``codes`` [rows, cols] (one byte each) and ``scales``
    [rows, ceil(cols / 32)] (uint8); ``format`` is "int8" or "e4m3"."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, format: str):
        if format not in _lib.CKPT8_FORMATS:
            raise ValueError(f"format must be one of {sorted(_lib.CKPT8_FORMATS)}, not {format!r}")
        if codes.dim() != 2 or codes.element_size() != 1:
            raise ValueError("codes must be [rows, cols] of one byte each")
        _checked("codes", codes, tuple(codes.shape), codes.dtype, codes.device)
        groups = -(-codes.shape[1] // _lib.KT_CKPT8_GROUP)
        _checked("scales", scales, (codes.shape[0], groups), torch.uint8, codes.device)
        self.codes, self.scales, self.format = codes, scales, format
        self.shape = tuple(codes.shape)
        self.fmt = _lib.CKPT8_FORMATS[format]
        self.c = _lib.kt_ckpt8(self.fmt, codes.data_ptr(), scales.data_ptr())


def checkpoint8_buffers(rows: int, cols: int, format: str = "int8", device="cuda") -> Checkpoint8:
    codes = torch.empty((rows, cols), dtype=torch.int8, device=device)
    scales = torch.empty((rows, -(-cols // _lib.KT_CKPT8_GROUP)), dtype=torch.uint8, device=device)
    return Checkpoint8(codes, scales, format)


def pack_checkpoint8(x: torch.Tensor, format: str = "int8", out: Optional[Checkpoint8] = None,
                     stream=None) -> Checkpoint8:
    """The bf16 rows ``x`` [rows, cols] as a checkpoint."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    _checked("x", x, tuple(x.shape), torch.bfloat16, x.device)
    rows, cols = x.shape
    if out is None:
        _gpu(x)
        groups = -(-cols // _lib.KT_CKPT8_GROUP)
        out = Checkpoint8(_empty((rows, cols), torch.int8, x.device, stream),
                          _empty((rows, groups), torch.uint8, x.device, stream), format)
    elif out.format != format or out.shape != (rows, cols) or out.codes.device != x.device:
        raise ValueError(f"out must be a {format} checkpoint of {(rows, cols)} on {x.device}")
    if _elsewhere(_gpu(x)):
        with torch.cuda.device(x.device):
            return pack_checkpoint8(x, format, out, stream)
    _lib.kt_ckpt8_pack(x, rows, cols, out.fmt, out.codes, out.scales, _handle(stream, x.device))
    return out


def unpack_checkpoint8(checkpoint: Checkpoint8, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The bf16 rows that a checkpoint stands for."""
    dev = checkpoint.codes.device
    _checked("out", out, checkpoint.shape, torch.bfloat16, dev)
    if _elsewhere(_gpu(checkpoint.codes)):
        with torch.cuda.device(dev):
            return unpack_checkpoint8(checkpoint, out, stream)
    if out is None:
        out = _empty(checkpoint.shape, torch.bfloat16, dev, stream)
    _lib.kt_ckpt8_unpack(checkpoint.codes, checkpoint.scales, *checkpoint.shape, checkpoint.fmt, out,
                         _handle(stream, dev))
    return out


class DeviceRouter:
    """Routing of tokens to experts from their logits: what gives the expert ids and route
    weights of a DeviceLayer, and takes its route-weight gradient back to the logits.
    ``bias`` [E] (fp32, or None) takes part in the choice alone."""

    def __init__(self, num_experts: int, top_k: int, score: str = "softmax", num_groups: int = 1, top_groups: int = 1,
                 group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
                 bias: Optional[torch.Tensor] = None):
        if score not in _lib.SCORES:
            raise ValueError(f"score must be one of {sorted(_lib.SCORES)}, not {score!r}")
        if bias is not None:
            _checked("bias", bias, (num_experts,), torch.float32, bias.device)
        self.num_experts, self.top_k, self.bias = num_experts, top_k, bias
        self._c = {dtype: _lib.kt_router(num_experts, top_k, num_groups, top_groups, group_top, _lib.SCORES[score],
                                         int(bool(renormalize)), float(scale), code)
                   for dtype, code in _TYPES.items()}

    def _logits(self, logits):
        if logits.dtype not in _TYPES:
            raise ValueError(f"logits must be torch.float32 or torch.bfloat16, not {logits.dtype}")
        if logits.dim() != 2:
            raise ValueError("logits must be [tokens, num_experts]")
        _checked("logits", logits, (logits.shape[0], self.num_experts), logits.dtype, logits.device)
        return logits.shape[0], logits.device

    def forward(self, logits, token_mask=None, expert_ids=None, route_weights=None, load=None, accumulate=False,
                stream=None):
        """(expert_ids [tokens, k] int64, route_weights [tokens, k] fp32).  token_mask [tokens]:
        bool or uint8, 0 for padding.  load [E] int32 receives the slots per expert."""
        tokens, dev = self._logits(logits)
        shape = (tokens, self.top_k)
        if token_mask is not None:
            _checked("token_mask", token_mask, (tokens,),
                     torch.bool if token_mask.dtype is torch.bool else torch.uint8, dev)
        _checked("expert_ids", expert_ids, shape, torch.int64, dev)
        _checked("route_weights", route_weights, shape, torch.float32, dev)
        _checked("load", load, (self.num_experts,), torch.int32, dev)
        if self.bias is not None and self.bias.device != dev:
            raise ValueError(f"the bias is on {self.bias.device}, the logits are on {dev}")
        if _elsewhere(_gpu(logits)):
            with torch.cuda.device(dev):
                return self.forward(logits, token_mask, expert_ids, route_weights, load, accumulate, stream)
        if expert_ids is None:
            expert_ids = _empty(shape, torch.int64, dev, stream)
        if route_weights is None:
            route_weights = _empty(shape, torch.float32, dev, stream)
        _lib.kt_router_fwd(self._c[logits.dtype], tokens, logits, self.bias, token_mask, expert_ids, route_weights, load,
                           accumulate, _handle(stream, dev))
        return expert_ids, route_weights

    def backward(self, logits, expert_ids, grad_route, grad_logits=None, stream=None):
        """The gradient of the logits from grad_route [tokens, k] (as DeviceLayer.backward fills it)."""
        tokens, dev = self._logits(logits)
        shape = (tokens, self.top_k)
        _checked("expert_ids", expert_ids, shape, torch.int64, dev)
        _checked("grad_route", grad_route, shape, torch.float32, dev)
        _checked("grad_logits", grad_logits, (tokens, self.num_experts), logits.dtype, dev)
        if _elsewhere(_gpu(logits)):
            with torch.cuda.device(dev):
                return self.backward(logits, expert_ids, grad_route, grad_logits, stream)
        if grad_logits is None:
            grad_logits = _empty((tokens, self.num_experts), logits.dtype, dev, stream)
        _lib.kt_router_bwd(self._c[logits.dtype], tokens, logits, expert_ids, grad_route, grad_logits,
                           _handle(stream, dev))
        return grad_logits

    def update_bias(self, load, rate, stream=None) -> None:
        """Moves the bias by ``rate`` towards balance: up for experts below the mean load, down above."""
        if self.bias is None:
            raise ValueError("this router has no bias")
        _checked("load", load, (self.num_experts,), torch.int32, self.bias.device)
        _gpu(self.bias)
        with torch.cuda.device(self.bias.device):
            _lib.kt_router_update_bias(self.bias, load, self.num_experts, rate, stream)


class DeviceLinear:
    """A dense layer act(x W^T + b) + residual with its gradients: the router's logits, a shared
    expert's products.  ``weight`` [out, in] bf16, ``bias`` [out] fp32 or None."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: str = "none"):
        if activation not in _lib.ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)}, not {activation!r}")
        if weight.dim() != 2:
            raise ValueError("weight must be [out_features, in_features]")
        _checked("weight", weight, tuple(weight.shape), torch.bfloat16, weight.device)
        _checked("bias", bias, (weight.shape[0],), torch.float32, weight.device)
        self.weight, self.bias, self.activation = weight, bias, activation
        self.out_features, self.in_features = weight.shape
        self.device = weight.device
        self.linear = _lib.make_linear(weight, bias, activation)

    def workspace(self, tokens: int) -> torch.Tensor:
        """Of forward() for up to so many tokens."""
        n = _lib.kt_linear_workspace_bytes(self.linear, tokens)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def backward_workspace(self, tokens: int, checkpoint: bool = True) -> torch.Tensor:
        """Of backward() for up to so many tokens.  checkpoint=False: for inputs given as rows only (smaller)."""
        n = _lib.kt_linear_bwd_workspace_bytes(self.linear, tokens, checkpoint)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def grad_buffers(self, fill: Optional[float] = None) -> Dict[str, torch.Tensor]:
        """fp32 gradients of the weight and, where the layer has one, the bias."""
        shapes = {"weight": (self.out_features, self.in_features)}
        if self.bias is not None:
            shapes["bias"] = (self.out_features,)
        if fill is None:
            return {n: torch.empty(s, dtype=torch.float32, device=self.device) for n, s in shapes.items()}
        return {n: torch.full(s, fill, dtype=torch.float32, device=self.device) for n, s in shapes.items()}

    def forward(self, x, workspace, residual=None, preact=None, output=None, dtype=torch.bfloat16, stream=None):
        """act(x W^T + b) + residual.  ``dtype`` is that of an output made here (bf16 or fp32); ``preact``
        [tokens, out] bf16, if given, receives x W^T + b for the backward."""
        if x.dim() != 2:
            raise ValueError("x must be [tokens, in_features]")
        tokens, dev = x.shape[0], self.device
        shape = (tokens, self.out_features)
        _checked("x", x, (tokens, self.in_features), torch.bfloat16, dev)
        _checked("residual", residual, shape, torch.bfloat16, dev)
        _checked("preact", preact, shape, torch.bfloat16, dev)
        kind = _TYPES.get(dtype if output is None else output.dtype)
        if kind is None:
            raise ValueError("the output must be torch.bfloat16 or torch.float32")
        if output is not None:
            _checked("output", output, shape, output.dtype, dev)
        if _elsewhere(_gpu(x)):
            with torch.cuda.device(dev):
                return self.forward(x, workspace, residual, preact, output, dtype, stream)
        _workspace(workspace, dev)
        if output is None:
            output = _empty(shape, dtype, dev, stream)
        _lib.kt_linear_fwd(self.linear, tokens, x, residual, output, kind, preact, workspace,
                           _handle(stream, dev))
        return output

    def backward(self, x, grad_output, workspace, grads, preact=None, grad_input=None, grad_residual=None,
                 accumulate=False, grad_scale=1.0, stream=None, need_input=True):
        """Gradients of forward(): returns grad_input = dz W + grad_residual (None without need_input) and
        fills ``grads`` (from grad_buffers(); an empty dict: none) by the window rule.  ``x`` is the bf16
        rows or their Checkpoint8; ``preact`` is what forward() wrote, for a layer with an activation."""
        dev, ckpt, rows = self.device, None, x
        if isinstance(x, Checkpoint8):
            if x.codes.device != dev:
                raise ValueError(f"the checkpoint must be on {dev}, not on {x.codes.device}")
            ckpt, rows = x.c, None
        if len(x.shape) != 2 or x.shape[1] != self.in_features:
            raise ValueError(f"x must be [tokens, {self.in_features}], not {tuple(x.shape)}")
        tokens = x.shape[0]
        shape = (tokens, self.out_features)
        _checked("x", rows, (tokens, self.in_features), torch.bfloat16, dev)
        if grad_output.dtype not in _TYPES:
            raise ValueError("grad_output must be torch.bfloat16 or torch.float32")
        _checked("grad_output", grad_output, shape, grad_output.dtype, dev)
        if self.activation == "none":
            preact = None
        _checked("preact", preact, shape, torch.bfloat16, dev)
        _checked("grad_residual", grad_residual, tuple(x.shape), torch.bfloat16, dev)
        _checked("grad_input", grad_input, tuple(x.shape), torch.bfloat16, dev)
        d_weight, d_bias = grads.get("weight"), grads.get("bias")
        _checked("grads['weight']", d_weight, (self.out_features, self.in_features), torch.float32, dev)
        _checked("grads['bias']", d_bias, (self.out_features,), torch.float32, dev)
        if _elsewhere(_gpu(grad_output)):
            with torch.cuda.device(dev):
                return self.backward(x, grad_output, workspace, grads, preact, grad_input, grad_residual, accumulate,
                                     grad_scale, stream, need_input)
        _workspace(workspace, dev)
        if grad_input is None and need_input:
            grad_input = _empty(tuple(x.shape), torch.bfloat16, dev, stream)
        _lib.kt_linear_bwd(self.linear, tokens, rows, ckpt, preact, grad_output, _TYPES[grad_output.dtype],
                           grad_residual, grad_input, d_weight, d_bias, accumulate, grad_scale, workspace,
                           _handle(stream, dev))
        return grad_input


# ---------------------------------------------------------------- what completes a step


class DeviceNorm:
    """The norms on both sides of a block, with the block's gate and scale and the residual stream:
    h = x + scale * gate * token_gate * n(branch), y = N(h) * weight + bias.  ``kind`` is "rms" or "layer";
    the vectors are fp32 [hidden] or None; ``branch_norm``: n is a norm too, with branch_weight and
    branch_bias."""

    def __init__(self, hidden: int, kind: str = "rms", eps: float = 1e-6, scale: float = 1.0,
                 weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, branch_norm: bool = False,
                 branch_weight: Optional[torch.Tensor] = None, branch_bias: Optional[torch.Tensor] = None,
                 gate: Optional[torch.Tensor] = None):
        if kind not in _lib.NORMS:
            raise ValueError(f"kind must be one of {sorted(_lib.NORMS)}, not {kind!r}")
        vectors = {"weight": weight, "bias": bias, "branch_weight": branch_weight, "branch_bias": branch_bias,
                   "gate": gate}
        given = [v for v in vectors.values() if v is not None]
        for name, v in vectors.items():
            if v is not None:
                _checked(name, v, (hidden,), torch.float32, given[0].device)
        self.hidden, self.kind, self.vectors = hidden, kind, vectors
        self.branch_norm = bool(branch_norm)
        self.device = given[0].device if given else None
        pointers = [None if v is None else v.data_ptr() for v in vectors.values()]
        self._c = {dtype: _lib.kt_norm(hidden, _lib.NORMS[kind], code, int(self.branch_norm), eps, scale, *pointers)
                   for dtype, code in _TYPES.items()}

    def _stream_type(self, name, x):
        """(tokens, device) of a tensor of the residual stream."""
        if x.dtype not in _TYPES:
            raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, not {x.dtype}")
        if x.dim() != 2:
            raise ValueError(f"{name} must be [tokens, {self.hidden}]")
        _checked(name, x, (x.shape[0], self.hidden), x.dtype, x.device if self.device is None else self.device)
        return x.shape[0], x.device

    def forward(self, x, branch=None, token_gate=None, h=None, y=None, need_h=True, need_y=True, stream=None):
        """(h, y) of the residual stream x [tokens, hidden] (bf16 or fp32) and a block's output ``branch``
        (bf16; without it h is x), token_gate [tokens] fp32.  ``h`` may be x itself; what is not needed is
        None."""
        tokens, dev = self._stream_type("x", x)
        shape = (tokens, self.hidden)
        _checked("branch", branch, shape, torch.bfloat16, dev)
        _checked("token_gate", token_gate, (tokens,), torch.float32, dev)
        _checked("h", h, shape, x.dtype, dev)
        _checked("y", y, shape, torch.bfloat16, dev)
        if branch is None and (h is not None or token_gate is not None):
            raise ValueError("h and token_gate need a branch (without it h is x)")
        if _elsewhere(_gpu(x)):
            with torch.cuda.device(dev):
                return self.forward(x, branch, token_gate, h, y, need_h, need_y, stream)
        if h is None and need_h and branch is not None:
            h = _empty(shape, x.dtype, dev, stream)
        if y is None and need_y:
            y = _empty(shape, torch.bfloat16, dev, stream)
        _lib.kt_norm_fwd(self._c[x.dtype], tokens, x, branch, token_gate, h, y, _handle(stream, dev))
        return x if branch is None else h, y

    def workspace(self, tokens: int, device=None) -> torch.Tensor:
        """Of backward() for up to so many tokens."""
        n = _lib.kt_norm_bwd_workspace_bytes(self._c[torch.bfloat16], tokens)
        return torch.empty(n, dtype=torch.uint8, device=device or self.device or "cuda")

    def grad_buffers(self, fill: Optional[float] = None, device=None) -> Dict[str, torch.Tensor]:
        """fp32 gradients of the vectors that the norms have."""
        new = torch.empty if fill is None else lambda *s, **k: torch.full(s, fill, **k)
        return {n: new(self.hidden, dtype=torch.float32, device=device or self.device)
                for n, v in self.vectors.items() if v is not None}

    def backward(self, h, workspace, grads, branch=None, token_gate=None, grad_h=None, grad_y=None, grad_x=None,
                 grad_branch=None, grad_token_gate=None, accumulate=False, grad_scale=1.0, need_input=True,
                 stream=None):
        """Gradients of forward() at its h, from grad_h (the residual stream's) and grad_y: returns
        (grad_x, grad_branch) and fills ``grads`` (from grad_buffers(); an empty dict: none) by the window
        rule and grad_token_gate [tokens] fp32.  grad_x may be grad_h itself.  need_input=False makes
        no grad_x and grad_branch beyond those given."""
        tokens, dev = self._stream_type("h", h)
        shape = (tokens, self.hidden)
        _checked("branch", branch, shape, torch.bfloat16, dev)
        _checked("token_gate", token_gate, (tokens,), torch.float32, dev)
        _checked("grad_h", grad_h, shape, h.dtype, dev)
        _checked("grad_y", grad_y, shape, torch.bfloat16, dev)
        _checked("grad_x", grad_x, shape, h.dtype, dev)
        _checked("grad_branch", grad_branch, shape, torch.bfloat16, dev)
        _checked("grad_token_gate", grad_token_gate, (tokens,), torch.float32, dev)
        for name in grads:
            if name not in self.vectors:
                raise ValueError(f"grads has no place for {name!r}")
            _checked(f"grads[{name!r}]", grads[name], (self.hidden,), torch.float32, dev)
        if _elsewhere(_gpu(h)):
            with torch.cuda.device(dev):
                return self.backward(h, workspace, grads, branch, token_gate, grad_h, grad_y, grad_x, grad_branch,
                                     grad_token_gate, accumulate, grad_scale, need_input, stream)
        _workspace(workspace, dev)
        if grad_x is None and need_input:
            grad_x = _empty(shape, h.dtype, dev, stream)
        if grad_branch is None and need_input and branch is not None:
            grad_branch = _empty(shape, torch.bfloat16, dev, stream)
        _lib.kt_norm_bwd(self._c[h.dtype], tokens, h, branch, token_gate, grad_h, grad_y, grad_x, grad_branch,
                         grad_token_gate, *(grads.get(n) for n in self.vectors), accumulate, grad_scale, workspace,
                         _handle(stream, dev))
        return grad_x, grad_branch


class DeviceAdamW:
    """AdamW over a dict of tensors (fp32 or bf16), all in one call.  No two of them share memory (tied weights stand
    in it once, with the sum of their gradients).

    ``states``: "fp32", or "e4m3" for 8-bit moments with one fp32 scale per 256 values.  ``master``: bf16
    tensors keep an fp32 copy that the updates are made to.  ``max_norm`` clips the gradients by their
    global norm; with it, or with ``check_finite``, the norm is computed (``grad_norm``), and one that is not
    finite leaves everything as it was.  ``no_decay``: names without weight decay.  ``state`` (as self.state)
    and ``step`` continue an earlier run; their tensors are used as they are.
    self.state[name] has m, v (with 8-bit states codes of m and of sqrt(v), and m_scale, v_scale) and master;
    self.step_count [1] int64 counts the steps on the GPU, so that a step in a graph can be replayed."""

    def __init__(self, params: Dict[str, torch.Tensor], lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, states: str = "fp32", master: bool = False,
                 max_norm: Optional[float] = None, check_finite: bool = False, no_decay=(), state=None, step=0):
        if states not in _lib.ADAMW_STATES:
            raise ValueError(f"states must be one of {sorted(_lib.ADAMW_STATES)}, not {states!r}")
        if not params:
            raise ValueError("params must hold a tensor")
        unknown = set(no_decay) - set(params)
        if unknown:
            raise ValueError(f"no_decay names no tensor of params: {sorted(unknown)}")
        self.params, self.states = dict(params), states
        self.device = dev = next(iter(params.values())).device
        self.lr, self.betas, self.eps, self.weight_decay, self.max_norm = lr, tuple(betas), eps, weight_decay, max_norm
        self.state = {}
        eight = states == "e4m3"
        for name, p in params.items():
            if p.dtype not in _TYPES:
                raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, not {p.dtype}")
            _checked(name, p, tuple(p.shape), p.dtype, dev)
            n = p.numel()
            have = dict((state or {}).get(name) or {})
            blocks = -(-n // _lib.KT_ADAMW_BLOCK)
            want = {"m": (torch.float8_e4m3fn if eight else torch.float32, (n,)),
                    "v": (torch.float8_e4m3fn if eight else torch.float32, (n,))}
            if eight:
                want.update(m_scale=(torch.float32, (blocks,)), v_scale=(torch.float32, (blocks,)))
            if master and p.dtype is torch.bfloat16:
                want["master"] = (torch.float32, tuple(p.shape))
            extra = set(have) - set(want)
            if extra:
                raise ValueError(f"state[{name!r}] has no place for {sorted(extra)}")
            for key, (dtype, shape) in want.items():
                t = have.get(key)
                if t is None:
                    t = p.detach().float() if key == "master" else torch.zeros(shape, dtype=dtype, device=dev)
                elif key in ("m", "v") and t.numel() == n and t.dim() != 1:
                    t = t.view(-1)
                _checked(f"state[{name!r}][{key!r}]", t, shape, dtype, dev)
                have[key] = t
            self.state[name] = have
        # all of them are updated at once: one that shares values with another would be updated twice, in no order
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), label) for name, p in params.items()
                       for label, t in ((repr(name), p), *((f"state[{name!r}][{k!r}]", s) for k, s in self.state[name].items()))
                       if t.numel())
        for (_, end, one), (begin, _, other) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError(f"{one} and {other} share memory: a tensor stands in params once")
        if isinstance(step, torch.Tensor):
            _checked("step", step, (1,), torch.int64, dev)
            self.step_count = step
        else:
            if step < 0:
                raise ValueError(f"step must not be negative, not {step}")
            self.step_count = torch.full((1,), int(step), dtype=torch.int64, device=dev)
        self.grad_norm = None
        if max_norm is not None or check_finite:
            self.grad_norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self._workspace = torch.empty(_lib.kt_adamw_workspace_bytes(len(params)), dtype=torch.uint8, device=dev)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._tensors = (_lib.kt_adamw_tensor * len(params))()
        for c, (name, p) in zip(self._tensors, params.items()):
            s = self.state[name]
            c.count, c.param_type, c.decay = p.numel(), _TYPES[p.dtype], int(name not in no_decay)
            c.param, c.master, c.m, c.v = ptr(p), ptr(s.get("master")), ptr(s["m"]), ptr(s["v"])
            c.m_scale, c.v_scale = ptr(s.get("m_scale")), ptr(s.get("v_scale"))
        self._slots = [(c, name, p.shape) for c, (name, p) in zip(self._tensors, params.items())]

    def step(self, grads: Dict[str, torch.Tensor], grad_scale: float = 1.0, lr: Optional[torch.Tensor] = None,
             stream=None) -> None:
        """One step from ``grads`` (a gradient, fp32 or bf16, for every name of params), times grad_scale.
        ``lr`` [1] fp32 on the GPU replaces self.lr, for schedules inside a graph.  Steps of one optimizer
        share its state and workspace: they run one after another."""
        dev = self.device
        for c, name, shape in self._slots:
            g = grads.get(name)
            if g is None:
                raise ValueError(f"grads has no {name!r}")
            kind = _TYPES.get(g.dtype)
            if kind is None:
                raise ValueError(f"grads[{name!r}] must be torch.float32 or torch.bfloat16, not {g.dtype}")
            if g.shape != shape or g.device != dev or not g.is_contiguous():
                _checked(f"grads[{name!r}]", g, shape, g.dtype, dev)
            c.grad, c.grad_type = g.data_ptr(), kind
        _checked("lr", lr, (1,), torch.float32, dev)
        if _elsewhere(_gpu(self.step_count)):
            with torch.cuda.device(dev):
                return self.step(grads, grad_scale, lr, stream)
        hyper = _lib.kt_adamw(self.lr, *self.betas, self.eps, self.weight_decay, self.max_norm or 0.0, grad_scale,
                              _lib.ADAMW_STATES[self.states])
        _lib.kt_adamw_step(hyper, self._tensors, len(self._tensors), self.step_count, self.grad_norm, lr,
                           self._workspace, _handle(stream, dev))
