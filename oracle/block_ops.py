"""Layer norm, the MoE gate with its balance loss, the combine of the experts' rows, their gradients and gradient
clipping, in 64 bits -- TEST INFRASTRUCTURE ONLY (see the package docstring).

Inputs are arrays of the values the library gets (bf16 and fp32 values are exact in float64); results are float64
before any rounding to the output's type.
"""

from __future__ import annotations

import numpy as np


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """x [M, N] -> (y, mean [M], rstd [M])."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """-> (dx, dweight, dbias), with the given mean and rstd."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    h = (x - mean) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def gate_probs(logits):
    """Row softmax; -inf gives 0, and a row of nothing but -inf zeros."""
    l = np.asarray(logits, np.float64)
    mx = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(mx), 0.0, mx))
    s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def moe_gate(logits, topk, renormalize=True, loss_coef=0.01, token_mask=None):
    """-> (ids [T, topk], weights, counts [E], loss)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    real = np.ones(T, bool) if token_mask is None else np.asarray(token_mask).astype(bool)
    p = gate_probs(l)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :topk]
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        s = w.sum(1, keepdims=True)
        w = np.divide(w, s, out=np.zeros_like(w), where=s != 0)
    w = np.where(real[:, None], w, 0.0)
    counts = np.bincount(ids[real].reshape(-1), minlength=E)
    tv = int(real.sum())
    loss = loss_coef * E * float((counts / (topk * tv) * p[real].sum(0) / tv).sum()) if tv else 0.0
    return ids, w, counts, loss


def moe_gate_backward(logits, ids, counts, dweights=None, dloss=None, renormalize=True, loss_coef=0.01,
                      token_mask=None):
    """-> dlogits [T, E]; the choice and the counts are constants."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    topk = ids.shape[1]
    real = np.ones(T, bool) if token_mask is None else np.asarray(token_mask).astype(bool)
    p = gate_probs(np.where(real[:, None], l, 0.0))
    tv = counts.sum() / topk
    g = np.zeros((T, E))
    if dloss is not None and tv > 0:
        g += float(dloss) * loss_coef * E * np.asarray(counts, np.float64) / (topk * tv * tv)
    if dweights is not None:
        dw = np.asarray(dweights, np.float64)
        if renormalize:
            sel = np.take_along_axis(p, ids, 1)
            s = sel.sum(1, keepdims=True)
            s = np.where(s == 0, np.inf, s)
            dw = (dw - (dw * sel / s).sum(1, keepdims=True)) / s
        np.add.at(g, (np.arange(T)[:, None], ids), dw)
    return np.where(real[:, None], p * (g - (g * p).sum(1, keepdims=True)), 0.0)


def moe_combine(D, entry_row, weights=None, residual=None):
    """-> out [T, N]."""
    D = np.asarray(D, np.float64)
    T, topk = entry_row.shape
    out = np.zeros((T, D.shape[1])) if residual is None else np.array(residual, np.float64)
    for t in range(T):
        for j in range(topk):
            if entry_row[t, j] >= 0:
                out[t] += (1.0 if weights is None else float(weights[t, j])) * D[entry_row[t, j]]
    return out


def moe_combine_backward(dout, D, entry_row, weights=None):
    """-> (dD [M, N], dweights [T, topk])."""
    dout, D = np.asarray(dout, np.float64), np.asarray(D, np.float64)
    T, topk = entry_row.shape
    dD, dw = np.zeros_like(D), np.zeros((T, topk))
    for t in range(T):
        for j in range(topk):
            r = entry_row[t, j]
            if r >= 0:
                dD[r] = (1.0 if weights is None else float(weights[t, j])) * dout[t]
                dw[t, j] = dout[t] @ D[r]
    return dD, dw


def clip_grad_norm(grads, max_norm, eps=1e-6):
    """-> (norm, the scaled gradients)."""
    norm = float(np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)))
    coef = min(1.0, max_norm / (norm + eps)) if norm + eps > 0 else 1.0
    return norm, [np.asarray(g, np.float64) * coef for g in grads]
