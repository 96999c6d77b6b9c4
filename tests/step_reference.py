"""Plain 64-bit implementations of the norms, of AdamW and of the experts for a
few tokens, and the error bounds that their fp32 computation may reach.

U is half a step of fp32 (2^-24), UB of bf16 (2^-8).  Sums of n products are held
to 8 sqrt(n) U times the sum of magnitudes, as in block_reference.  Errors
are carried through products and quotients to first order, and 1.1 covers the rest.
"""

import math

import numpy as np
import torch

from tests.block_reference import U, UB

F64 = torch.float64


def rounding(dtype):
    return UB if dtype is torch.bfloat16 else U


def _d(t):
    return None if t is None else t.detach().double().cpu()


class Norm:
    """N(v) of the rows of v, known to dv: value, its error, 1 / deviation and that one's relative error."""

    def __init__(self, v, dv, kind, eps):
        n = v.shape[1]
        sq = 8 * math.sqrt(n) * U
        c, dc = v, dv
        if kind == "layer":
            c = v - v.mean(1, keepdim=True)
            dc = dv + dv.mean(1, keepdim=True) + sq * v.abs().mean(1, keepdim=True) + 2 * U * (v.abs() + v.mean(1, keepdim=True).abs())
        var = (c * c).mean(1, keepdim=True) + eps
        self.r = 1 / torch.sqrt(var)
        # (the mean of squares: a sum of positive terms; then the mean, eps, root and quotient)
        self.rho = (2 * c.abs() * dc + dc * dc).mean(1, keepdim=True) / (2 * var) + sq / 2 + 6 * U
        self.v = c * self.r
        self.dv = 1.1 * (self.r * dc + self.v.abs() * (self.rho + 2 * U))


def _affine(v, dv, w, c):
    if w is not None:
        v, dv = v * w, dv * w.abs() + U * (v * w).abs()
    if c is not None:
        v = v + c
        dv = dv + U * v.abs()
    return v, dv


def norm_fwd(x, branch=None, token_gate=None, kind="rms", eps=1e-6, scale=1.0, weight=None, bias=None, branch_norm=False,
             branch_weight=None, branch_bias=None, gate=None):
    """(h, bound of h, y, bound of y) before the rounding to the outputs' type."""
    x, b, tg = _d(x), _d(branch), _d(token_gate)
    w, c, bw, bc, gate = map(_d, (weight, bias, branch_weight, branch_bias, gate))
    h, dh = x, torch.zeros_like(x)
    if b is not None:
        n, dn = b, torch.zeros_like(b)
        if branch_norm:
            s = Norm(b, dn, kind, eps)
            n, dn = _affine(s.v, s.dv, bw, bc)
        by = scale * (1 if gate is None else gate) * (1 if tg is None else tg[:, None])
        z = by * n
        h = x + z
        dh = 1.1 * torch.as_tensor(by).abs() * dn + 4 * U * z.abs() + U * h.abs()
    s = Norm(h, dh, kind, eps)
    y, dy = _affine(s.v, s.dv, w, c)
    return h, dh, y, dy


def _norm_bwd(a, da, s, kind):
    """The gradient through a Norm from a, known to da, and its error."""
    n = a.shape[1]
    sq = 8 * math.sqrt(n) * U
    m1, dm1 = torch.zeros(a.shape[0], 1, dtype=F64), torch.zeros(a.shape[0], 1, dtype=F64)
    if kind == "layer":
        m1 = a.mean(1, keepdim=True)
        dm1 = da.mean(1, keepdim=True) + sq * a.abs().mean(1, keepdim=True)
    m2 = (a * s.v).mean(1, keepdim=True)
    dm2 = (a.abs() * s.dv + s.v.abs() * da).mean(1, keepdim=True) + (sq + 4 * U) * (a * s.v).abs().mean(1, keepdim=True)
    inner = a - m1 - s.v * m2
    d = da + dm1 + s.v.abs() * dm2 + m2.abs() * s.dv + 4 * U * (a.abs() + m1.abs() + (s.v * m2).abs())
    return s.r * inner, 1.1 * (s.r * d + (s.rho + 2 * U) * (s.r * inner).abs())


def norm_bwd(h, branch=None, token_gate=None, grad_h=None, grad_y=None, kind="rms", eps=1e-6, scale=1.0, weight=None, bias=None,
             branch_norm=False, branch_weight=None, branch_bias=None, gate=None):
    """{name: (gradient, bound)}: x, branch, token_gate, and the vectors' by their names."""
    h, b, tg, gh, gy = map(_d, (h, branch, token_gate, grad_h, grad_y))
    w, bw, bc, gate = map(_d, (weight, branch_weight, branch_bias, gate))
    zero = torch.zeros_like(h)
    rows = 8 * math.sqrt(h.shape[0] + 1) * U
    out = {}
    d, dd = zero, zero
    if gy is not None:
        s = Norm(h, zero, kind, eps)
        a = gy if w is None else gy * w
        d, dd = _norm_bwd(a, U * a.abs(), s, kind)
        out["weight"] = (gy * s.v).sum(0), (gy.abs() * s.dv).sum(0) + rows * (gy * s.v).abs().sum(0)
        out["bias"] = gy.sum(0), rows * gy.abs().sum(0)
    if gh is not None:
        d = d + gh
        dd = dd + U * d.abs()
    out["x"] = d, dd
    if b is None:
        return out
    n, dn = b, zero
    if branch_norm:
        s = Norm(b, zero, kind, eps)
        n, dn = _affine(s.v, s.dv, bw, bc)
    t = scale if tg is None else scale * tg[:, None]
    p = d * n
    dp = n.abs() * dd + d.abs() * dn + 3 * U * p.abs()
    ts = torch.as_tensor(t, dtype=F64).abs()
    out["gate"] = (t * p).sum(0), (ts * dp).sum(0) + rows * (ts * p.abs()).sum(0)
    g = 1.0 if gate is None else gate
    ga = torch.as_tensor(g, dtype=F64).abs()
    cols = 8 * math.sqrt(h.shape[1] + 1) * U
    out["token_gate"] = scale * (g * p).sum(1), abs(scale) * ((ga * dp).sum(1) + (cols + 4 * U) * (ga * p.abs()).sum(1))
    e = t * g * d
    de = ts * ga * dd + 4 * U * e.abs()
    if branch_norm:
        out["branch_weight"] = (e * s.v).sum(0), (e.abs() * s.dv + s.v.abs() * de).sum(0) + rows * (e * s.v).abs().sum(0)
        out["branch_bias"] = e.sum(0), de.sum(0) + rows * e.abs().sum(0)
        if bw is not None:
            e, de = e * bw, de * bw.abs() + U * (e * bw).abs()
        e, de = _norm_bwd(e, de, s, kind)
    out["branch"] = e, de
    return out


# ---------------------------------------------------------------- AdamW


def e4m3_step(w):
    """The distance of E4M3 numbers at w (a hair above, so that a value just below a power of two counts as above it)."""
    return torch.exp2(torch.floor(torch.log2((w.abs() * (1 + 2.0**-18)).clamp(min=2.0**-6))) - 3)


def e4m3_blocks(v, dv, root):
    """(codes' values, scales, bounds of both) of v, known to dv, in blocks of 256."""
    n = v.numel()
    pad = torch.cat([v, v.new_zeros(-n % 256)]).view(-1, 256)
    dpad = torch.cat([dv, dv.new_zeros(-n % 256)]).view(-1, 256)
    amax = pad.abs().amax(1, keepdim=True)
    some = amax >= 2.0**-100
    w = torch.where(some, pad / torch.where(some, amax, 1.0) * 448, 0.0)
    step = e4m3_step(w)
    q = torch.round(w / step) * step
    if root:
        q = torch.where((w > 0) & (q < 2.0**-9), 2.0**-9, q)
    scale = torch.where(some, amax / 448, 0.0)[:, 0]
    # a block's largest is known to its largest dv; a value then moves against it, and may round to the next code
    most = 1.1 * dpad.amax(1, keepdim=True) / torch.where(some, amax, 1.0)
    dw = 448 * 1.1 * dpad / torch.where(some, amax, 1.0) + w.abs() * (most + 4 * U)
    return q.view(-1)[:n], scale, torch.where(dw > 0, step + dw, 0.0).view(-1)[:n], scale * (most[:, 0] + 4 * U)


def adamw(p, grad, m, v, t, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, mult=1.0):
    """(p, m, v) of step t and their bounds; mult: what multiplies the gradient."""
    p, m, v = _d(p), _d(m), _d(v)
    g = _d(grad) * mult
    b1, b2 = betas
    mm = (b1 * m).abs() + ((1 - b1) * g).abs()
    m, dm = b1 * m + (1 - b1) * g, 4 * U * mm
    v = b2 * v + (1 - b2) * g * g
    dv = 8 * U * v
    size = lr / (1 - b1**t)
    den = torch.sqrt(v) / math.sqrt(1 - b2**t) + eps
    up = size * m / den
    new = p * (1 - lr * weight_decay) - up
    dp = 3 * U * p.abs() + 20 * U * up.abs() + 1.1 * size * dm / den + 2.0**-148
    return (new, dp), (m, dm + 2.0**-148), (v, dv + 2.0**-147)


# ---------------------------------------------------------------- experts


E2M1 = torch.tensor([s * x for s in (1, -1) for x in (0, 0.5, 1, 1.5, 2, 3, 4, 6)], dtype=F64)


def weights(packed, scale, fmt):
    """(dequantised rows, the magnitudes that the kernels' sums have) in 64 bits."""
    c = torch.stack([packed & 15, packed >> 4], -1).flatten(1).long()
    s = scale.double().repeat_interleave(32, 1)
    if fmt == "mxfp4":
        w = E2M1.to(c.device)[c] * s
        return w, w.abs()
    # sums of (1 + c / 16) x and 3/2 x, 16 s times
    return (c - 8) * s, (16 + c + 24) * s.abs()


def experts(x, ids, rw, layer, fmt="rawint4", limit=0.0, lora=None, sc=0.0):
    """(output, bound before its rounding); layer: the packed and scale tensors by name."""
    x, rw = _d(x), _d(rw)
    e_count = layer["gate_packed"].shape[0]
    out, bound = torch.zeros_like(x), torch.zeros_like(x)

    def product(name, e, v, dv, split):  # split: what v is rounded by before the product
        w, mag = weights(layer[name + "_packed"][e].cpu(), layer[name + "_scale"][e].cpu(), fmt)
        n = v.numel()
        y = w @ v
        d = w.abs() @ (dv + split * v.abs()) + 8 * math.sqrt(2 * n) * U * (mag @ v.abs())
        if lora is not None:
            a, b = lora[name + "_lora_a"][e].double().cpu(), lora[name + "_lora_b"][e].double().cpu()
            t = a @ v
            dt = a.abs() @ dv + 8 * math.sqrt(n) * U * (a.abs() @ v.abs())
            y = y + sc * (b @ t)
            d = d + abs(sc) * (b.abs() @ dt + (8 * math.sqrt(a.shape[0]) + 4) * U * (b.abs() @ t.abs()))
        return y, d + 2 * U * y.abs()

    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < e_count:
                continue
            v = x[t]
            g, dg = product("gate", e, v, torch.zeros_like(v), 0.0)
            u, du = product("up", e, v, torch.zeros_like(v), 0.0)
            if limit > 0:
                g, u = g.clamp(max=limit), u.clamp(-limit, limit)
            silu = g / (1 + torch.exp(-g))
            h = silu * u
            dh = 1.1 * (1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du) + 16 * U * (1 + g.abs()) * h.abs()
            y, dy = product("down", e, h, dh, 2.0**-11)
            out[t] += rw[t, j] * y
            bound[t] += rw[t, j].abs() * (dy + 2 * U * y.abs())
    return out, 1.1 * bound + 8 * U * out.abs()


def rel_l2(actual, expected):
    a, e = actual.double().cpu(), expected.double().cpu()
    return float((a - e).norm() / e.norm()) if float(e.norm()) else float(np.abs(a).max())
