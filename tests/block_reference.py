"""Plain 64-bit implementations of the operators around the experts, and the
error bounds that their fp32 / bf16 computation may reach.

U is half a step of fp32 (2^-24), UB of bf16 (2^-8).  Sums of n fp32 products
are held to 8 sqrt(n) U times the sum of magnitudes (the probabilistic bound
of Higham and Mary, SIAM J. Sci. Comput. 41(5), 2019, Theorem 2.4, with lambda
= 8), which holds for any order of summation.
"""

import math

import numpy as np
import torch

U = 2.0**-24
UB = 2.0**-8


def rounding(dtype):
    return {torch.float32: U, torch.bfloat16: UB}[dtype]


def within(tag, actual, expected, bound):
    """Every |actual - expected| <= bound; both may be infinite or NaN at the same places."""
    a = actual.detach().double().cpu().numpy()
    e = expected.double().cpu().numpy() if torch.is_tensor(expected) else np.asarray(expected, np.float64)
    b = bound.double().cpu().numpy() if torch.is_tensor(bound) else np.asarray(bound, np.float64)
    assert a.shape == e.shape, f"{tag}: {a.shape} against {e.shape}"
    assert np.array_equal(np.isnan(a), np.isnan(e)), f"{tag}: NaNs at other places"
    fine = np.isfinite(e)
    assert np.array_equal(a[~fine & ~np.isnan(e)], e[~fine & ~np.isnan(e)]), f"{tag}: infinities at other places"
    b = np.broadcast_to(b, a.shape)
    off = np.abs(a[fine] - e[fine])
    bad = ~(off <= b[fine])
    worst = float(np.max(off / np.maximum(b[fine], 1e-300))) if off.size else 0.0
    print(f"{tag}: {worst:.3f} of the bound", flush=True)
    assert not bad.any(), f"{tag}: {int(bad.sum())} of {off.size} values off by up to {worst:.2f} times the bound"


# ---------------------------------------------------------------- routing


def scores(logits, score):
    l = np.asarray(logits, np.float64)
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = l.max(1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            e = np.exp(l - m)
            z = e.sum(1, keepdims=True)
            return np.where(z > 0, e / np.where(z > 0, z, 1), np.where(np.isnan(z), np.nan, 0.0))
        return 1.0 / (1.0 + np.exp(-l))


def undefined_rows(logits, score, bias=None):
    l = np.asarray(logits, np.float64)
    bad = np.isnan(l).any(1)
    if score == "softmax":
        bad |= np.isposinf(l).any(1)
    if bias is not None and (np.isnan(bias).any() or np.isposinf(bias).any()):
        bad[:] = True
    return bad


def route(logits, top_k, score="softmax", num_groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0,
          bias=None, mask=None):
    """(ids, weights, load) by one stable sort per token."""
    l = np.asarray(logits, np.float64)
    t, e = l.shape
    s = scores(l, score)
    bad = undefined_rows(l, score, bias)
    ids = np.full((t, top_k), -1, np.int64)
    w = np.zeros((t, top_k))
    per = e // num_groups
    for i in range(t):
        if mask is not None and not mask[i]:
            continue
        if bad[i]:
            ids[i] = np.arange(top_k)
            w[i] = np.nan
            continue
        b = np.zeros(e) if bias is None else np.asarray(bias, np.float64)
        c = np.where(np.isneginf(l[i]) | np.isneginf(b), -np.inf, s[i] + b)
        if num_groups > 1:
            by = l[i] if bias is None and group_top == 1 else c
            g = np.sort(by.reshape(num_groups, per), 1)[:, ::-1][:, :group_top].sum(1)
            kept = np.argsort(-g, kind="stable")[:top_groups]
            c = np.where(np.isin(np.arange(e) // per, kept), c, -np.inf)
        if bias is None:  # s is monotone in the logit, also where it saturates in 64 bits
            c = np.where(c > -np.inf, l[i], -np.inf)
        order = np.argsort(-c, kind="stable")[:top_k]
        order = order[c[order] > -np.inf]
        n = len(order)
        ids[i, :n] = order
        total = s[i, order].sum() + 1e-20 if renormalize else 1.0
        w[i, :n] = scale * s[i, order] / total
    load = np.bincount(ids[ids >= 0], minlength=e)
    return ids, w, load


def route_precision(logits):
    """Relative error of a score, a weight or one of their sums in fp32: the exponential's argument l - m is
    rounded (U |l - m|), and some thirty roundings follow (the exponential, a tree of sums, the quotients)."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isfinite(l), l, 0.0)
    return U * (40 + 2 * (l.max(1) - l.min(1)) + 2 * np.abs(l).max(1))


def route_bwd(logits, ids, g, score="softmax", renormalize=True, scale=1.0):
    """(dlogits, bound of an fp32 computation before its rounding to the result's type)."""
    l = np.asarray(logits, np.float64)
    t, e = l.shape
    s = scores(l, score)
    bad = undefined_rows(l, score)
    out, bound = np.zeros((t, e)), np.zeros((t, e))
    prec = route_precision(l)
    for i in range(t):
        use = [j for j in range(ids.shape[1]) if 0 <= ids[i, j] < e]
        if not use:
            continue
        if bad[i]:
            out[i] = np.nan
            continue
        at, gi = ids[i, use], np.asarray(g[i], np.float64)[use]
        si = s[i, at]
        ds, mag = np.zeros(e), np.zeros(e)
        if renormalize:
            total = si.sum() + 1e-20
            d = (gi * si).sum() / total
            dmag = (np.abs(gi) * si).sum() / total
            np.add.at(ds, at, scale * (gi - d) / total)
            np.add.at(mag, at, abs(scale) * (np.abs(gi) + dmag) / total)
        else:
            np.add.at(ds, at, scale * gi)
            np.add.at(mag, at, abs(scale) * np.abs(gi))
        if score == "softmax":
            # with renormalisation sum ds s cancels to 1e-20 / S of its terms
            dot = (scale * d * 1e-20 / total) if renormalize else (ds * s[i]).sum()
            # d = sum g p may cancel: its error is prec * sum |g| p, however small d itself is
            dot_mag = abs(scale) * dmag * 1e-20 / total if renormalize else (mag * s[i]).sum()
            out[i] = s[i] * (ds - dot)
            # a score below fp32's normal range is held in steps of 2^-149, and meets 1 / S up to 1e20 in mag
            bound[i] = (4 * prec[i] * s[i] + 2.0**-147) * (mag + dot_mag)
        else:
            out[i] = ds * s[i] * (1 - s[i])
            # 1 - s is a difference: its error is U, not U (1 - s)
            bound[i] = 4 * prec[i] * mag * s[i] * ((1 - s[i]) + 2 * U)
            bound[i] += 4 * U * mag * s[i]
    return out, bound


# ---------------------------------------------------------------- checkpoints


def checkpoint(x, fmt):
    """Values on the grid of every group, NaN where a group holds an infinity or a NaN."""
    x = np.asarray(x, np.float64)
    out = np.zeros_like(x)
    for c in range(0, x.shape[1], 32):
        v = x[:, c:c + 32]
        for i in range(v.shape[0]):
            a = np.abs(v[i]).max()
            if not np.isfinite(v[i]).all():
                out[i, c:c + 32] = np.nan
                continue
            if a == 0:
                continue
            e = -127
            if fmt == "int8":
                while np.rint(math.ldexp(a, -e)) > 127 and e < 121:
                    e += 1
                out[i, c:c + 32] = np.ldexp(np.clip(np.rint(np.ldexp(v[i], -e)), -127, 127), e)
            else:
                while math.ldexp(a, -e) > 448:
                    e += 1
                w = np.ldexp(v[i], -e)
                ex = np.floor(np.log2(np.maximum(np.abs(w), 2.0**-6)))
                q = np.rint(w / 2.0 ** (ex - 3)) * 2.0 ** (ex - 3)
                out[i, c:c + 32] = np.ldexp(np.clip(q, -240, 240) if e == 120 else q, e)
    return out


# ---------------------------------------------------------------- dense products


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))
    return z


def act_grad(z, name):
    z = z.clone().requires_grad_()
    (g,) = torch.autograd.grad(act(z, name).sum(), z)
    return g


def linear(x, w, bias=None, residual=None, name="none"):
    """(y, z, bound of y, bound of z) before the rounding to the outputs' type."""
    x, w = x.double().cpu(), w.double().cpu()
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double().cpu()
        mag = mag + bias.double().cpu().abs()
    zb = 8 * math.sqrt(x.shape[1] + 1) * U * mag
    y = act(z, name)
    # every activation's slope is below 1.13; its own evaluation takes about ten roundings of z's size
    yb = 1.13 * zb + (16 * U * z.abs() if name != "none" else 0)
    if residual is not None:
        y = y + residual.double().cpu()
        yb = yb + U * y.abs()
    return y, z, yb, zb


def linear_bwd(x, w, dy, z=None, grad_residual=None, name="none"):
    """{"dx", "dw", "db"} and their bounds before the results' own rounding."""
    x, w, dy = x.double().cpu(), w.double().cpu(), dy.cpu()
    exact_dz = name == "none" and dy.dtype is torch.bfloat16
    dy = dy.double()
    slope = act_grad(z.double().cpu(), name) if name != "none" else torch.ones_like(dy)
    dz = dy * slope
    # the slope's evaluation: about 24 roundings of terms of size up to 1.2
    eval_err = 32 * U * dy.abs() * 1.2 if name != "none" else torch.zeros_like(dy)
    out, bound = {}, {}
    out["dx"] = dz @ w
    dx_dz = eval_err + (0 if exact_dz else UB * dz.abs())
    bound["dx"] = dx_dz @ w.abs() + 8 * math.sqrt(w.shape[0] + 1) * U * (dz.abs() @ w.abs())
    if grad_residual is not None:
        out["dx"] = out["dx"] + grad_residual.double().cpu()
        bound["dx"] = bound["dx"] + U * out["dx"].abs()
    out["dw"] = dz.t() @ x
    # two bf16 planes hold a dz to 2^-8 of 2^-8
    dw_dz = eval_err + (0 if exact_dz else UB * UB * dz.abs())
    n = (1 if exact_dz else 2) * x.shape[0]
    bound["dw"] = dw_dz.t() @ x.abs() + 8 * math.sqrt(n + 1) * U * (dz.abs().t() @ x.abs())
    out["db"] = dz.sum(0)
    bound["db"] = eval_err.sum(0) + 8 * math.sqrt(x.shape[0] + 1) * U * dz.abs().sum(0)
    return out, bound
