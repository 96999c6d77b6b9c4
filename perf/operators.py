"""The operators around the routed experts, as measured: routing, dense products with an epilogue, 8-bit activation checkpoints.

``run`` computes each operator in plain torch operations; with ``own`` set it calls the library instead.  ``exact`` computes the
same outputs in 64 bits, written apart from the plain form.
"""

import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")
LARGEST = 8192 * 7168 * 2048  # tokens x in x out of the largest product


def listed():
    return [
        # the gate projection of one decoded token, 384 experts over a hidden size of 7168: latency
        {"name": "logits_1", "op": "linear", "tokens": 1, "k": 7168, "n": 384, "act": "none", "bias": False, "residual": False, "preact": False, "fp32": True},
        # the gate projection of a long training batch
        {"name": "logits_16384", "op": "linear", "tokens": 16384, "k": 7168, "n": 384, "act": "none", "bias": False, "residual": False, "preact": False, "fp32": True},
        # a dense (shared) expert's second product, ragged token count, everything in the epilogue, kept for a backward
        {"name": "dense_4001_all", "op": "linear", "tokens": 4001, "k": 2048, "n": 7168, "act": "gelu_tanh", "bias": True, "residual": True, "preact": True, "fp32": False},
        # the gate projection's backward: fp32 gradient of the logits, dx added to the experts' grad_input
        {"name": "logits_bwd_4096", "op": "linear_bwd", "tokens": 4096, "k": 7168, "n": 384, "act": "none", "bias": False, "residual": True, "fp32": True, "ckpt": "none"},
        # a dense (shared) expert's first product backward from an 8-bit checkpoint of its input: the largest product here
        {"name": "dense_bwd_8192_ckpt", "op": "linear_bwd", "tokens": 8192, "k": 7168, "n": 2048, "act": "silu", "bias": True, "residual": False, "fp32": False, "ckpt": "int8"},
        # routing of one decoded token: sigmoid scores, balance bias, 4 of 8 groups
        {"name": "route_1", "op": "route", "tokens": 1, "experts": 384, "top_k": 8, "score": "sigmoid", "groups": 8, "top_groups": 4, "group_top": 2, "bias": True, "renorm": True, "scale": 2.5, "bf16": False, "mask": False, "load": False},
        # a training batch, softmax scores of bf16 logits, padded tokens, expert load counted
        {"name": "route_4096_softmax", "op": "route", "tokens": 4096, "experts": 384, "top_k": 8, "score": "softmax", "groups": 1, "top_groups": 1, "group_top": 1, "bias": False, "renorm": False, "scale": 1.0, "bf16": True, "mask": True, "load": True},
        # a long training batch with balance bias and groups
        {"name": "route_16384_groups", "op": "route", "tokens": 16384, "experts": 384, "top_k": 8, "score": "sigmoid", "groups": 8, "top_groups": 4, "group_top": 2, "bias": True, "renorm": True, "scale": 2.5, "bf16": False, "mask": False, "load": False},
        # the routing gradient of a training batch, both score functions
        {"name": "route_bwd_4096", "op": "route_bwd", "tokens": 4096, "experts": 384, "top_k": 8, "score": "sigmoid", "renorm": True, "scale": 2.5, "bf16": False},
        {"name": "route_bwd_16384", "op": "route_bwd", "tokens": 16384, "experts": 384, "top_k": 8, "score": "softmax", "renorm": True, "scale": 1.0, "bf16": True},
        # a layer's input kept in 8 bits and read back: a small batch, and a long one
        {"name": "ckpt_32_e4m3", "op": "ckpt", "tokens": 32, "k": 7168, "format": "e4m3"},
        {"name": "ckpt_16384_int8", "op": "ckpt", "tokens": 16384, "k": 7168, "format": "int8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "linear_bwd", "route", "route", "route_bwd", "ckpt"))
    if op in ("linear", "linear_bwd"):
        while True:
            t, k, n = _log(rng, 1, 16384), 8 * _log(rng, 8, 896), _log(rng, 1, 7168)
            if t * k * n <= LARGEST:
                break
        c = {"op": op, "tokens": t, "k": k, "n": n, "act": rng.choice(ACTIVATIONS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "fp32": rng.random() < 0.4}
        if op == "linear":
            c["preact"] = rng.random() < 0.5
        else:
            c["ckpt"] = rng.choice(("none", "none", "int8", "e4m3"))
        return c
    if op == "ckpt":
        return {"op": op, "tokens": _log(rng, 1, 16384), "k": _log(rng, 8, 7168), "format": rng.choice(("int8", "e4m3"))}
    groups = rng.choice((1, 1, 2, 4, 8)) if op == "route" else 1
    per = max(2, _log(rng, 4, 512) // groups)
    experts = groups * per
    top_groups = rng.randint(1, groups)
    top_k = rng.randint(1, min(12, top_groups * per))
    c = {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "top_k": top_k, "score": rng.choice(("softmax", "sigmoid")), "renorm": rng.random() < 0.6, "scale": rng.choice((1.0, 2.5)), "bf16": rng.random() < 0.4}
    if op == "route_bwd" and top_k == 1:
        c["renorm"] = False  # one expert's renormalised weight is constant: its gradient is the 1e-20's alone
    if op == "route":
        c.update(groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)), bias=rng.random() < 0.6, mask=rng.random() < 0.4, load=rng.random() < 0.4)
    return c


def work(case):
    t = case["tokens"]
    if case["op"] == "ckpt":
        return {"bytes": t * case["k"] * (2 + 2 + 2 * (1 + 1 / 32)), "flops": 4.0 * t * case["k"]}
    if case["op"] in ("linear", "linear_bwd"):
        k, n = case["k"], case["n"]
        y = 4 if case["fp32"] else 2
        if case["op"] == "linear":
            b = 2 * t * k + 2 * n * k + t * n * (y + 2 * case["residual"] + 2 * case["preact"]) + 4 * n * case["bias"]
            return {"bytes": b, "flops": 2.0 * t * k * n}
        x = 2 if case["ckpt"] == "none" else 1 + 1 / 32
        b = t * k * (x + 2 + 2 * case["residual"]) + 2 * n * k + 4 * n * k + t * n * (y + 2 * (case["act"] != "none")) + 4 * n * case["bias"]
        return {"bytes": b, "flops": 4.0 * t * k * n}
    e, k, w = case["experts"], case["top_k"], 2 if case["bf16"] else 4
    if case["op"] == "route":
        return {"bytes": t * e * w + t * k * 12 + 4 * e * case["bias"] + t * case["mask"] + 4 * e * case["load"], "flops": 10.0 * t * e}
    return {"bytes": 2 * t * e * w + t * k * 12, "flops": 8.0 * t * e}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    t, s = case["tokens"], {"case": case}
    if case["op"] == "ckpt":
        # hidden states: a few channels are much larger than the rest
        x = normal(t, case["k"], dtype=F32)
        x *= torch.exp(normal(case["k"], std=0.7, dtype=F32))
        s["x"] = x.to(BF16)
        return s
    if case["op"] in ("linear", "linear_bwd"):
        k, n = case["k"], case["n"]
        s["x"] = normal(t, k)
        s["weight"] = normal(n, k, std=k**-0.5)
        s["bias"] = normal(n, dtype=F32) if case["bias"] else None
        if case["op"] == "linear":
            s["residual"] = normal(t, n) if case["residual"] else None
            return s
        s["preact"] = normal(t, n) if case["act"] != "none" else None
        s["dy"] = normal(t, n, dtype=F32 if case["fp32"] else BF16)
        s["residual"] = normal(t, k) if case["residual"] else None
        if case["ckpt"] != "none":
            s["codes"], s["scales"] = _pack(s.pop("x"), case["ckpt"])
        return s
    e = case["experts"]
    s["logits"] = normal(t, e, std=1.5, dtype=BF16 if case["bf16"] else F32)
    if case["op"] == "route":
        s["bias"] = normal(e, std=0.1, dtype=F32) if case["bias"] else None
        s["mask"] = torch.rand(t, generator=g, device=DEV) < 0.9 if case["mask"] else None
        return s
    s["ids"] = torch.rand(t, e, generator=g, device=DEV).argsort(1)[:, : case["top_k"]].contiguous()
    s["grad_route"] = normal(t, case["top_k"], dtype=F32)
    return s


# ---------------------------------------------------------------- the plain forms


def _act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5**0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z**3)))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5**0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        a = (2 / math.pi) ** 0.5
        th = torch.tanh(a * (z + 0.044715 * z**3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * a * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _groups(x):
    """Rows as groups of 32 columns, the last one filled up with zeros."""
    t, k = x.shape
    pad = -k % 32
    if pad:
        x = torch.cat([x, x.new_zeros(t, pad)], 1)
    return x.reshape(t, -1, 32)


def _pow2(e):
    """2^e exactly, -127 <= e <= 127 (a power function may be a rounding off)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(F32)


def _pack(x, fmt):
    """8-bit codes [tokens, k] and one exponent byte per 32 columns: the value is code * 2^(byte - 127)."""
    t, k = x.shape
    v = _groups(x.float())
    amax = v.abs().amax(2)
    frac, exp = torch.frexp(amax)  # amax = frac * 2^exp, frac in [0.5, 1)
    if fmt == "int8":
        e = exp - 7 + (frac * 128 >= 127.5)
    else:
        e = exp - 9 + (frac > 0.875)
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    v = v * _pow2(-e.unsqueeze(2))
    v = torch.round(v).to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn).view(torch.int8)
    return v.reshape(t, -1)[:, :k].contiguous(), (e + 127).to(torch.uint8)


def _unpack(codes, scales, fmt):
    v = codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    e = scales.to(torch.int32).repeat_interleave(32, 1)[:, : codes.shape[1]] - 127
    return v * _pow2(e)


def _plain_linear(s, case):
    z = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y if case["fp32"] else y.to(BF16)}
    if case["preact"]:
        out["z"] = z.to(BF16)
    return out


def _plain_linear_bwd(s, case):
    x = s["x"].float() if case["ckpt"] == "none" else _unpack(s["codes"], s["scales"], case["ckpt"])
    dz = s["dy"].float()
    if s["preact"] is not None:
        dz = dz * _act_grad(s["preact"].float(), case["act"])
    dx = dz @ s["weight"].float()
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    out = {"dx": dx.to(BF16), "dw": dz.t() @ x}
    if s["bias"] is not None:
        out["db"] = dz.sum(0)
    return out


def _plain_route(s, case):
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    logits = s["logits"].float()
    score = torch.softmax(logits.double(), 1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-logits.double()))
    choice = score if s["bias"] is None else score + s["bias"].double()  # 64 bits: experts may lie next to each other
    if case["groups"] > 1:
        top = choice.view(t, case["groups"], -1).sort(dim=2, descending=True).values[:, :, : case["group_top"]].sum(2)
        kept = top.sort(dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros(t, case["groups"], dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(e // case["groups"], 1), choice, -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k].contiguous()
    if case["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = w * case["scale"]
    if s["mask"] is not None:
        ids = torch.where(s["mask"][:, None], ids, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    out = {"ids": ids, "w": w}
    if case["load"]:
        out["load"] = (torch.bincount(ids.flatten() + 1, minlength=e + 1)[1:]).to(torch.int32)
    return out


def _plain_route_bwd(s, case):
    logits, g = s["logits"].float(), s["grad_route"]
    if case["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    chosen = p.gather(1, s["ids"])
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True) + 1e-20
        ds = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    else:
        ds = g
    ds = torch.zeros_like(p).scatter_(1, s["ids"], ds * case["scale"])
    dl = p * (ds - (ds * p).sum(1, keepdim=True)) if case["score"] == "softmax" else ds * p * (1 - p)
    return {"dlogits": dl.to(s["logits"].dtype)}


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "linear":
        return _plain_linear(state, case)
    if case["op"] == "linear_bwd":
        return _plain_linear_bwd(state, case)
    if case["op"] == "route":
        return _plain_route(state, case)
    if case["op"] == "route_bwd":
        return _plain_route_bwd(state, case)
    codes, scales = _pack(state["x"], case["format"])
    return {"x": _unpack(codes, scales, case["format"]).to(BF16)}


# ---------------------------------------------------------------- the library's calls


def _own(s, case):
    from int4_quantized_moe_amd import device

    op, t = case["op"], case["tokens"]
    kept = s.get("kept")  # the handle, workspace and output buffers that a program keeps
    if kept is None:
        kept = s["kept"] = {}
        if op in ("linear", "linear_bwd"):
            k, n = case["k"], case["n"]
            h = kept["h"] = device.DeviceLinear(s["weight"], s["bias"], case["act"])
            if op == "linear":
                kept["ws"] = h.workspace(t)
                kept["y"] = torch.empty(t, n, dtype=F32 if case["fp32"] else BF16, device=DEV)
                kept["z"] = torch.empty(t, n, dtype=BF16, device=DEV) if case["preact"] else None
            else:
                kept["ws"] = h.backward_workspace(t)
                kept["dx"] = torch.empty(t, k, dtype=BF16, device=DEV)
                kept["grads"] = h.grad_buffers()
                kept["x"] = s["x"] if case["ckpt"] == "none" else device.Checkpoint8(s["codes"], s["scales"], case["ckpt"])
        elif op == "ckpt":
            kept["ck"] = device.checkpoint8_buffers(t, case["k"], case["format"], DEV)
            kept["x"] = torch.empty_like(s["x"])
        else:
            more = {} if op == "route_bwd" else {"num_groups": case["groups"], "top_groups": case["top_groups"], "group_top": case["group_top"], "bias": s["bias"]}
            kept["h"] = device.DeviceRouter(case["experts"], case["top_k"], score=case["score"], renormalize=case["renorm"], scale=case["scale"], **more)
            if op == "route":
                kept["ids"] = torch.empty(t, case["top_k"], dtype=torch.int64, device=DEV)
                kept["w"] = torch.empty(t, case["top_k"], dtype=F32, device=DEV)
                kept["load"] = torch.empty(case["experts"], dtype=torch.int32, device=DEV) if case["load"] else None
            else:
                kept["dl"] = torch.empty_like(s["logits"])
    if op == "linear":
        kept["h"].forward(s["x"], kept["ws"], residual=s["residual"], preact=kept["z"], output=kept["y"])
        return {"y": kept["y"], "z": kept["z"]} if case["preact"] else {"y": kept["y"]}
    if op == "linear_bwd":
        kept["h"].backward(kept["x"], s["dy"], kept["ws"], kept["grads"], preact=s["preact"], grad_input=kept["dx"], grad_residual=s["residual"])
        out = {"dx": kept["dx"], "dw": kept["grads"]["weight"]}
        return {**out, "db": kept["grads"]["bias"]} if case["bias"] else out
    if op == "route":
        kept["h"].forward(s["logits"], token_mask=s["mask"], expert_ids=kept["ids"], route_weights=kept["w"], load=kept["load"])
        out = {"ids": kept["ids"], "w": kept["w"]}
        return {**out, "load": kept["load"]} if case["load"] else out
    if op == "route_bwd":
        kept["h"].backward(s["logits"], s["ids"], s["grad_route"], grad_logits=kept["dl"])
        return {"dlogits": kept["dl"]}
    device.pack_checkpoint8(s["x"], case["format"], kept["ck"])
    device.unpack_checkpoint8(kept["ck"], kept["x"])
    return {"x": kept["x"]}


# ---------------------------------------------------------------- in 64 bits


def _phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


_EXACT = {
    "none": (lambda z: z, lambda z: torch.ones_like(z)),
    "relu": (lambda z: z * (z > 0), lambda z: (z > 0).double()),
    "silu": (lambda z: z * torch.sigmoid(z), lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)),
    "gelu": (lambda z: z * _phi(z), lambda z: _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)),
    # 0.5 (1 + tanh u) = sigmoid(2u)
    "gelu_tanh": (
        lambda z: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z * z * z)),
        lambda z: torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z * z * z))
        + z
        * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z * z * z))
        * torch.sigmoid(-math.sqrt(8 / math.pi) * (z + 0.044715 * z * z * z))
        * math.sqrt(8 / math.pi)
        * (1 + 0.134145 * z * z),
    ),
}


def _exact_pow2(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _floor_log2(v):
    return (v.view(torch.int64) >> 52) - 1023


def _exact_checkpoint(x, fmt):
    """Every group's values on the grid its largest magnitude gives."""
    x = x.double()
    out = torch.zeros_like(x)
    for c in range(0, x.shape[1], 32):
        v = x[:, c : c + 32]
        amax = v.abs().max(1, keepdim=True).values
        floor = _floor_log2(torch.where(amax > 0, amax, 1.0))
        if fmt == "int8":
            step = _exact_pow2(floor - 6)
            step = torch.where(amax / step >= 127.5, 2 * step, step)
            out[:, c : c + 32] = torch.round(v / step) * step
        else:
            unit = _exact_pow2(floor - 8)
            unit = torch.where(amax / unit > 448, 2 * unit, unit)
            w = v / unit
            # three mantissa bits above 2^-6, the spacing of 2^-6 below it
            step = _exact_pow2(_floor_log2(w.abs().clamp(min=2.0**-6)) - 3)
            out[:, c : c + 32] = torch.round(w / step) * step * unit
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "ckpt":
        return {"x": _exact_checkpoint(s["x"], case["format"])}
    if op == "linear":
        z = torch.mm(s["x"].double(), s["weight"].double().transpose(0, 1))
        z = z if s["bias"] is None else z + s["bias"].double()
        y = _EXACT[case["act"]][0](z)
        y = y if s["residual"] is None else y + s["residual"].double()
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    if op == "linear_bwd":
        if case["ckpt"] == "none":
            x = s["x"].double()
        else:
            v = s["codes"].double() if case["ckpt"] == "int8" else s["codes"].view(torch.float8_e4m3fn).double()
            x = v * _exact_pow2(s["scales"].int() - 127).repeat_interleave(32, 1)[:, : case["k"]]
        dz = s["dy"].double()
        dz = dz if s["preact"] is None else dz * _EXACT[case["act"]][1](s["preact"].double())
        dx = torch.mm(dz, s["weight"].double())
        dx = dx if s["residual"] is None else dx + s["residual"].double()
        out = {"dx": dx, "dw": torch.mm(dz.transpose(0, 1).contiguous(), x)}
        return {**out, "db": dz.sum(0)} if case["bias"] else out
    logits = s["logits"].double()
    p = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        c = p.clone() if s["bias"] is None else p + s["bias"].double()
        rows = torch.arange(t, device=DEV)
        if case["groups"] > 1:
            left = c.view(t, case["groups"], -1).clone()
            sums = torch.zeros(t, case["groups"], dtype=F64, device=DEV)
            for _ in range(case["group_top"]):
                best, at = left.max(2)
                sums += best
                left.scatter_(2, at.unsqueeze(2), -math.inf)
            dropped = torch.ones(t, case["groups"], dtype=torch.bool, device=DEV)
            for _ in range(case["top_groups"]):
                at = sums.max(1).indices
                dropped[rows, at] = False
                sums[rows, at] = -math.inf
            c[dropped.unsqueeze(2).expand(t, case["groups"], e // case["groups"]).reshape(t, e)] = -math.inf
        w = torch.zeros(t, k, dtype=F64, device=DEV)
        for j in range(k):
            at = c.max(1).indices
            w[:, j] = p[rows, at]
            c[rows, at] = -math.inf
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        w = w * case["scale"]
        if s["mask"] is not None:
            w[~s["mask"]] = 0
        out = {"ids": None, "w": w}
        return {**out, "load": None} if case["load"] else out
    # the gradient of scale * p_i / sum p by automatic differentiation
    leaf = logits.clone().requires_grad_()
    p = torch.softmax(leaf, 1) if case["score"] == "softmax" else torch.sigmoid(leaf)
    w = p.gather(1, s["ids"])
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    (dl,) = torch.autograd.grad((w * s["grad_route"].double()).sum() * case["scale"], leaf)
    return {"dlogits": dl}
