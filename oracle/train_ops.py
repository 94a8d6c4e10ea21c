"""The router with bias and expert groups, the RMS norms around a block, the gated activation, their gradients and AdamW,
in 64 bits -- TEST INFRASTRUCTURE ONLY (see the package docstring).

Inputs are arrays of the values the library gets (bf16 and fp32 values are exact in float64); results are float64
before any rounding to the output's type.  AdamW's 8-bit states are codes, and so are formed with the roundings that the
interface names, in float32.
"""

from __future__ import annotations

import numpy as np

from .e4m3 import e4m3_decode, e4m3_encode
from .block_ops import gate_probs


def route_scores(logits, score="sigmoid"):
    l = np.asarray(logits, np.float64)
    if score == "softmax":
        return gate_probs(l)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def moe_route(logits, topk, bias=None, score="sigmoid", groups=1, topk_groups=1, renormalize=True, scale=1.0,
              token_mask=None):
    """-> (ids [T, topk], weights, counts [E])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    real = np.ones(T, bool) if token_mask is None else np.asarray(token_mask).astype(bool)
    s = route_scores(l, score)
    out = np.isneginf(l) | np.isneginf(b)
    with np.errstate(invalid="ignore"):
        c = np.where(out, -np.inf, s + b)
    c = np.where(np.isnan(c), np.inf, c)
    two = -np.sort(-c.reshape(T, groups, E // groups), axis=2)[:, :, :2]
    best = two[:, :, 0] if two.shape[2] == 1 else np.where(np.isneginf(two[:, :, 1]), two[:, :, 0], two.sum(2))
    rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
    keep = np.repeat(rank < topk_groups, E // groups, axis=1)
    order = c if bias is not None else np.where(out, -np.inf, np.where(np.isnan(l), np.inf, l))
    # what is ruled out comes behind everything that is not, and what is not kept behind that
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -order, ~keep), axis=1)[:, :topk]
    w = np.where(np.take_along_axis(out, ids, 1), 0.0, np.take_along_axis(s, ids, 1))
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total != 0)
    w = np.where(real[:, None], w * scale, 0.0)
    return ids, w, np.bincount(ids[real].reshape(-1), minlength=E)


def moe_route_backward(logits, ids, dweights, score="sigmoid", renormalize=True, scale=1.0, token_mask=None):
    """-> dlogits; ids outside [0, E) have no part."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids = np.asarray(ids)
    inside = (ids >= 0) & (ids < E)
    at = np.where(inside, ids, 0)
    s = route_scores(l, score)
    d = np.where(inside, np.asarray(dweights, np.float64) * scale, 0.0)
    sel = np.where(inside, np.take_along_axis(s, at, 1), 0.0)
    if renormalize:
        total = sel.sum(1, keepdims=True)
        by = np.divide(1.0, total, out=np.zeros_like(total), where=total != 0)
        d = np.where(inside, (d - (d * sel).sum(1, keepdims=True) * by) * by, 0.0)
    G = np.zeros((T, E))
    np.add.at(G, (np.arange(T)[:, None], at), d)
    if score == "sigmoid":
        dl = G * s * route_scores(-l, "sigmoid")
    else:
        dl = s * (G - (G * s).sum(1, keepdims=True))
    return dl if token_mask is None else np.where(np.asarray(token_mask).astype(bool)[:, None], dl, 0.0)


def _one(w, n):
    return np.ones(n) if w is None else np.asarray(w, np.float64)


def residual_rms_norm(x, f=None, weight=None, gate=None, scale=1.0, post_norm=False, post_weight=None, eps=1e-6):
    """-> (h, y, rstd, rstd_f or None)."""
    h = np.asarray(x, np.float64)
    n = h.shape[1]
    rstd_f = None
    if f is not None:
        u = np.asarray(f, np.float64)
        if post_norm:
            rstd_f = 1.0 / np.sqrt((u * u).mean(1) + eps)
            u = u * rstd_f[:, None] * _one(post_weight, n)
        h = h + scale * _one(gate, n) * u
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, h * rstd[:, None] * _one(weight, n), rstd, rstd_f


def residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f=None, weight=None, gate=None, scale=1.0, post_norm=False,
                               post_weight=None):
    """-> (dx, df, dweight, dgate, dpost), with the given statistics."""
    some = h if h is not None else dh
    n = np.shape(some)[1]
    dx = np.zeros(np.shape(some)) if dh is None else np.asarray(dh, np.float64)
    dw = None
    if dy is not None:
        dy, r = np.asarray(dy, np.float64), np.asarray(rstd, np.float64)[:, None]
        e = np.asarray(h, np.float64) * r
        g = dy * _one(weight, n)
        dx = dx + r * (g - e * (g * e).mean(1, keepdims=True))
        dw = (dy * e).sum(0)
    if f is None:
        return dx, None, dw, None, None
    k = np.asarray(f, np.float64)
    q = dx * scale * _one(gate, n) * _one(post_weight, n)
    df = q
    if post_norm:
        rf = np.asarray(rstd_f, np.float64)[:, None]
        k = k * rf
        df = rf * (q - k * (q * k).mean(1, keepdims=True))
    S = scale * (dx * k).sum(0)
    return dx, df, dw, S * _one(post_weight, n), S * _one(gate, n)


def swiglu(gu):
    """[M, 2F] -> h [M, F]."""
    gu = np.asarray(gu, np.float64)
    F = gu.shape[-1] // 2
    return gu[..., :F] * route_scores(gu[..., :F]) * gu[..., F:]


def swiglu_backward(dh, gu):
    gu, dh = np.asarray(gu, np.float64), np.asarray(dh, np.float64)
    F = gu.shape[-1] // 2
    g, u = gu[..., :F], gu[..., F:]
    s, rest = route_scores(g), route_scores(-g)
    return np.concatenate([dh * u * s * (1.0 + g * rest), dh * g * s], -1)


# ------------------------------------------------------------------ AdamW

def adamw(p, g, m, v, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, coef=1.0):
    """One step, the t-th, in 64 bits -> (p, m, v)."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * coef
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    return p - lr * (weight_decay * p + (m / (1.0 - beta1 ** t)) / (np.sqrt(v / (1.0 - beta2 ** t)) + eps)), m, v


def state_values(codes, scales):
    """What 8-bit states stand for, in float32 as the step reads them."""
    n = codes.size
    return e4m3_decode(codes).astype(np.float32) * np.repeat(np.asarray(scales, np.float32), 128)[:n]


def adamw_states(g, m, v_root, beta1, beta2, coef=1.0):
    """The new m and root of v in float32, each product and sum rounded."""
    f = np.float32
    g = np.asarray(g, f) * f(coef)
    m = f(beta1) * np.asarray(m, f) + f(1.0 - beta1) * g
    r = np.asarray(v_root, f)
    return m, np.sqrt(f(beta2) * (r * r) + (f(1.0 - beta2) * g) * g)


def encode_states(x, t, root):
    """The codes and scales of 8-bit states after step t; root: second moments' roots."""
    f = np.float32
    x = np.asarray(x, f)
    n = x.size
    b = np.zeros((n + 127) // 128 * 128, f)
    b[:n] = x
    b = b.reshape(-1, 128)
    top = np.abs(b).max(1)
    live = top >= f(2.0 ** -60)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(live, f(448) * (f(1) / top), f(0))
    scale = np.where(live, top * (f(1) / f(448)), f(0)).astype(f)
    y = (np.abs(b) * inv[:, None]).astype(f).astype(np.float64)
    place = np.arange(b.size, dtype=np.uint64).reshape(b.shape)
    z = np.uint64(1 << 31) if root else np.uint64(0)
    u = (place * np.uint64(0xC13FA9A9) + np.uint64(t) * np.uint64(0x91E10DA5) + z) & np.uint64(0xFFFFFFFF)
    u = (u >> np.uint64(12)).astype(np.float64) / 2 ** 20
    unit = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    c = np.minimum(np.floor(y / unit + u) * unit, 448.0)
    if root:
        c = np.where((b > 0) & live[:, None], np.maximum(c, 2.0 ** -9), c)
    c = np.copysign(c, b).reshape(-1)[:n]
    return e4m3_encode(c), scale
