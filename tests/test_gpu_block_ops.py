"""The training operators on the GPU against the 64-bit oracle: every type, odd and one-element sizes, strides,
unaligned tensors, masks that leave nothing, infinities and NaN in masked places, other streams and graphs.

Tolerances are error bounds of the formulas.  With u = 2^-24 (one fp32 rounding), a sum of n terms in which
each thread adds L of them one after another and the threads' sums join in a tree is off by at most (L + 12) u times
the sum of the terms' magnitudes; each further operation adds u.  A bf16 result adds its own rounding, 2^-8 of its
value at most (half a unit in the last of 8 bits, and as much again where the fp32 value crosses a midpoint).
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import block_ops as ob
from tests.gpu_util import check_status, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _draw(shape, dtype, seed, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda") * std + mean).to(DT[dtype])


def _np(t):
    return t.detach().double().cpu().numpy()


def _within(got, want, bound, dtype, what):
    """|got - want| <= bound (fp32 errors) plus the rounding of the result's type."""
    got = _np(got)
    assert got.shape == want.shape, what
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    tol = bound + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0.0) + 1e-37
    bad = np.abs(got - want) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - want) / tol), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bounds; worst at {i}: got {got[i]}, "
                             f"want {want[i]}, tolerance {tol[i]}")


def _strided(shape, dtype, pad, offset, seed=None, **kw):
    """A matrix with `pad` more elements a row in memory, starting `offset` elements into its buffer."""
    M, N = shape
    buf = torch.full((M * (N + pad) + offset + 8,), float("nan"), dtype=DT[dtype], device="cuda")
    t = buf[offset: offset + M * (N + pad)].view(M, N + pad)[:, :N]
    if seed is not None:
        t.copy_(_draw(shape, dtype, seed, **kw))
    return t, buf


# ------------------------------------------------------------------ layer norm

def _norm_bounds(x, w, b, mean, rstd, N):
    """Bounds of y: the mean's error is (L + 12) u mean|x|, rstd's relative error (L + 16) u, and the difference,
    two products and the sum round once each."""
    k = (N / 256 + 16) * U
    ax = np.abs(x)
    spread = (ax + np.abs(mean)[:, None] + 2 * ax.mean(1, keepdims=True)) * rstd[:, None]
    return 2 * k * (spread * (np.abs(w) if w is not None else 1.0) + (np.abs(b) if b is not None else 0.0))


NORM_SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 31), (3, 64), (7, 127), (130, 128), (3, 129), (9, 264), (2, 1000),
              (33, 1024), (2, 1025), (3, 2048), (5, 4099), (4, 4096), (3, 7168), (161, 7168), (2, 8200), (3, 16384),
              (2, 20001), (2, 40000), (1, 70008)]


@pytest.mark.parametrize("M,N", NORM_SIZES)
@pytest.mark.parametrize("xd,yd,wd", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f32", "bf16", "f32"),
                                      ("bf16", "f32", "f32")])
def test_layer_norm_and_gradients(M, N, xd, yd, wd):
    x, w, b = _draw((M, N), xd, 1, 2.0, 0.5), _draw((N,), wd, 2, 0.3, 1.0), _draw((N,), wd, 3)
    y, mean, rstd = g.layer_norm(x, w, b, out_dtype=DT[yd])
    xn, wn, bn = _np(x), _np(w), _np(b)
    ry, rmean, rrstd = ob.layer_norm(xn, wn, bn)
    k = (N / 256 + 16) * U
    _within(mean, rmean, k * np.abs(xn).mean(1), "f32", "mean")
    # rstd moves by half of the variance's relative error; with eps the variance is at least 1e-5
    var_err = 2 * k * ((np.abs(xn) + np.abs(rmean)[:, None]) ** 2).mean(1) * rrstd ** 2
    _within(rstd, rrstd, (k + var_err) * rrstd, "f32", "rstd")
    bound = _norm_bounds(xn, wn, bn, rmean, rrstd, N) + np.abs(ry) * var_err[:, None]
    _within(y, ry, bound, yd, "y")

    dy = _draw((M, N), yd, 4, 0.1)
    dx, dw, db = g.layer_norm_backward(dy, x, w, mean, rstd)
    _check_norm_grads(dx, dw, db, dy, x, w, mean, rstd, xd)
    dx2, dw2, db2 = g.layer_norm_backward(dy, x, w, mean, rstd)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)  # the same bits again
    only, none_w, none_b = g.layer_norm_backward(dy, x, w, mean, rstd, weight_grads=False)
    assert torch.equal(only, dx) and none_w is None and none_b is None


def _check_norm_grads(dx, dw, db, dy, x, w, mean, rstd, xd):
    M, N = x.shape
    xn, dyn, mu, r = _np(x), _np(dy), _np(mean)[:, None], _np(rstd)[:, None]
    wn = None if w is None else _np(w)
    rdx, rdw, rdb = ob.layer_norm_backward(dyn, xn, wn, _np(mean), _np(rstd))
    gw = np.abs(dyn) * (1.0 if wn is None else np.abs(wn))
    hb = (np.abs(xn) + np.abs(mu)) * r  # bounds |h| and, times u, its rounding
    k = (N / 256 + 20) * U
    bound = 2 * k * r * (gw + gw.mean(1, keepdims=True) + hb * (gw * hb).mean(1, keepdims=True))
    _within(dx, rdx, bound, xd, "dx")
    kr = (min(M, 304) + M / 304 + 20) * U  # rows one after another, then the partial rows
    _within(dw, rdw, kr * (np.abs(dyn) * hb).sum(0), "f32", "dweight")
    _within(db, rdb, kr * np.abs(dyn).sum(0), "f32", "dbias")


@pytest.mark.parametrize("N", [8, 1000, 1024, 4096, 7168, 10000])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (1, 3)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_layer_norm_strides_and_alignment(N, pad, offset, xd):
    M = 5
    x, _ = _strided((M, N), xd, pad, offset, 5)
    y, ybuf = _strided((M, N), xd, pad, offset)
    w = _draw((N + 3,), xd, 6)[3:]  # an unaligned weight
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    g.fp8g_layer_norm(x, w, None, y, mean, rstd)
    ry, rmean, rrstd = ob.layer_norm(_np(x), _np(w))
    _within(y, ry, _norm_bounds(_np(x), _np(w), None, rmean, rrstd, N) + 1e-5 * np.abs(ry), xd, "y")
    assert int(torch.isnan(ybuf).sum()) == ybuf.numel() - M * N  # nothing but the rows was written
    dy, _ = _strided((M, N), xd, pad, offset, 7)
    dx, dxbuf = _strided((M, N), xd, pad, offset)
    dw, db = torch.empty(N + 1, device="cuda")[1:], torch.empty(N, device="cuda")
    g.fp8g_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db)
    _check_norm_grads(dx, dw, db, dy, x, w, mean, rstd, xd)
    assert int(torch.isnan(dxbuf).sum()) == dxbuf.numel() - M * N


@pytest.mark.parametrize("N", [64, 1000, 7168])
def test_layer_norm_without_weights_and_in_place(N):
    x = _draw((6, N), "f32", 8)
    want = ob.layer_norm(_np(x))[0]
    bound = _norm_bounds(_np(x), None, None, *ob.layer_norm(_np(x))[1:], N) + 1e-5 * np.abs(want)
    y = g.layer_norm(x)[0]
    g.fp8g_layer_norm(x, None, None, x)  # y is x; no statistics
    assert torch.equal(x, y)
    _within(y, want, bound, "f32", "y")
    mean, rstd = x.mean(1).contiguous(), torch.ones(6, device="cuda")
    dy = _draw((6, N), "f32", 9)
    dx, dw, db = g.layer_norm_backward(dy, x, None, mean, rstd)
    _check_norm_grads(dx, dw, db, dy, x, None, mean, rstd, "f32")


@pytest.mark.parametrize("N", [32, 1024, 4099, 7168])
def test_layer_norm_constant_rows_large_means_and_bad_rows(N):
    x = _draw((5, N), "f32", 10)
    x[0] = 3.5                 # no spread: y = bias, rstd = 1 / sqrt(eps)
    x[1] += 10000.0            # a mean far above the spread
    x[2, N // 2] = float("nan")
    x[3, 0] = float("inf")
    y, mean, rstd = g.layer_norm(x)
    # the constant's mean is off by at most k |x|, and y by that times rstd
    k = (N / 256 + 16) * U
    assert float(y[0].abs().max()) <= 2 * k * 3.5 * 1e-5 ** -0.5
    xn = _np(x)
    ry, rmean, rrstd = ob.layer_norm(xn[[1, 4]])
    var_err = 2 * k * (np.abs(xn[[1, 4]]).mean(1) * k * rrstd) ** 2 + 4 * k
    bound = _norm_bounds(xn[[1, 4]], None, None, rmean, rrstd, N) + np.abs(ry) * var_err[:, None]
    _within(y[[1, 4]], ry, bound, "f32", "rows beside bad ones")
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).any())


def test_layer_norm_no_rows():
    x = torch.empty((0, 64), device="cuda")
    y, mean, rstd = g.layer_norm(x)
    assert y.shape == (0, 64) and mean.numel() == 0
    dx, dw, db = g.layer_norm_backward(x, x, None, mean, rstd)
    assert not dw.any() and not db.any()


def test_layer_norm_many_short_rows():
    M, N = 20011, 96
    x, dy, w = _draw((M, N), "bf16", 11), _draw((M, N), "bf16", 12, 0.1), _draw((N,), "f32", 13)
    y, mean, rstd = g.layer_norm(x, w)
    ry, rmean, rrstd = ob.layer_norm(_np(x), _np(w))
    _within(y, ry, _norm_bounds(_np(x), _np(w), None, rmean, rrstd, N) + 1e-5 * np.abs(ry), "bf16", "y")
    dx, dw, db = g.layer_norm_backward(dy, x, w, mean, rstd)
    _check_norm_grads(dx, dw, db, dy, x, w, mean, rstd, "bf16")


# many rows a resident CTA, so that its ring of row stages goes round many times; the last ones have a ring of two
# stages, and rows that two CTAs share
@pytest.mark.parametrize("M,N,xd,yd", [(3001, 1032, "bf16", "bf16"), (4000, 2048, "f32", "bf16"),
                                       (2500, 7168, "bf16", "bf16"), (3000, 1531, "bf16", "bf16"),
                                       (2000, 5003, "f32", "f32"), (1300, 8190, "bf16", "f32"),
                                       (1500, 16384, "f32", "f32"), (1111, 12001, "bf16", "bf16"),
                                       (5000, 1020, "bf16", "bf16"), (9000, 333, "f32", "bf16")])
def test_layer_norm_many_rows(M, N, xd, yd):
    x, dy, w = _draw((M, N), xd, 15, 1.0, 0.3), _draw((M, N), yd, 16, 0.1), _draw((N,), "f32", 17)
    y, mean, rstd = g.layer_norm(x, w, out_dtype=DT[yd])
    ry, rmean, rrstd = ob.layer_norm(_np(x), _np(w))
    k = (N / 256 + 16) * U
    _within(mean, rmean, k * np.abs(_np(x)).mean(1), "f32", "mean")
    _within(y, ry, _norm_bounds(_np(x), _np(w), None, rmean, rrstd, N) + 4 * k * np.abs(ry), yd, "y")
    dx, dw, db = g.layer_norm_backward(dy, x, w, mean, rstd)
    _check_norm_grads(dx, dw, db, dy, x, w, mean, rstd, xd)
    check_status()  # no wait ran out
    # a row's result does not depend on how many rows the call has (here: rows on the 16-byte grid)
    if N % 8 == 0:
        assert torch.equal(g.layer_norm(x[-5:], w, out_dtype=DT[yd])[0], y[-5:])
        assert torch.equal(g.layer_norm_backward(dy[-5:], x[-5:], w, mean[-5:], rstd[-5:])[0], dx[-5:])


# ------------------------------------------------------------------ gate

def _gate_k(E, spread):
    """Roundings of a probability: its exponent's argument (|l - max| u of it), the exponential (2), the sum."""
    return (E / 32 + 24 + spread) * U


def _check_gate(logits, topk, renorm, mask, coef=0.05):
    T, E = logits.shape
    ids, w, counts, loss = g.moe_gate(logits, topk, renormalize=renorm, loss_coef=coef, token_mask=mask)
    ln = _np(logits)
    mn = None if mask is None else mask.cpu().numpy()
    rids, rw, rcounts, rloss = ob.moe_gate(ln, topk, renorm, coef, mn)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.array_equal(counts.cpu().numpy(), rcounts)
    finite = ln[np.isfinite(ln)]
    k = _gate_k(E, finite.max() - finite.min() if finite.size else 0.0)
    _within(w, rw, 2 * k * rw, "f32", "weights")
    # the loss's terms are all positive; each expert's sum is over T rows at most
    _within(loss, np.array([rloss]), np.array([(k + (T / 8 + 350) * U) * abs(rloss)]), "f32", "loss")
    dw = torch.randn((T, topk), generator=_gen(20), device="cuda")
    dloss = torch.full((1,), 1.5, device="cuda")
    xd = "bf16" if logits.dtype == torch.bfloat16 else "f32"
    for d1, d2 in ((dw, dloss), (dw, None), (None, dloss)):
        dl = g.moe_gate_backward(logits, ids, counts, d1, d2, renormalize=renorm, loss_coef=coef, token_mask=mask)
        args = (None if d1 is None else _np(d1), None if d2 is None else 1.5, renorm, coef, mn)
        want = ob.moe_gate_backward(ln, rids, rcounts, *args)
        bound = _gate_grad_bound(ln, rids, rcounts, *args) * 3 * k
        _within(dl, want, bound, xd, "dlogits")
    return ids, w, counts, loss


def _gate_grad_bound(ln, ids, counts, dw, dloss, renorm, coef, mn):
    """The sum of the magnitudes that make up dlogits."""
    real = np.ones(len(ln), bool) if mn is None else mn.astype(bool)
    p = ob.gate_probs(np.where(real[:, None], ln, 0.0))
    E, topk = ln.shape[1], ids.shape[1]
    tv = max(counts.sum() / topk, 1)
    G = np.zeros_like(p)
    if dloss is not None:
        G += dloss * coef * E * counts / (topk * tv * tv)
    if dw is not None:
        a = np.abs(dw)
        if renorm:
            sel = np.take_along_axis(p, ids, 1)
            s = sel.sum(1, keepdims=True)
            s = np.where(s == 0, np.inf, s)
            a = 2 * (a + (a * sel / s).sum(1, keepdims=True)) / s
        np.add.at(G, (np.arange(len(p))[:, None], ids), a)
    return np.where(real[:, None], p * (G + (G * p).sum(1, keepdims=True)), 0.0)


@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 2, 2), (3, 4, 1), (5, 7, 7), (64, 8, 2), (33, 16, 4), (17, 31, 3),
                                      (64, 32, 8), (65, 33, 2), (100, 48, 6), (40, 64, 8), (9, 100, 8), (257, 128, 4),
                                      (300, 160, 6), (2500, 256, 8), (31, 257, 9), (19, 384, 32), (12, 512, 8),
                                      (5, 1000, 10), (4, 2048, 32), (5000, 8, 2), (4999, 64, 1)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("renorm,masked", [(True, False), (False, True)])
def test_gate_and_gradient(T, E, topk, xd, renorm, masked):
    logits = _draw((T, E), xd, T + E, 1.5)
    mask = (torch.arange(T, device="cuda") % 7 != 3) if masked else None
    a = _check_gate(logits, topk, renorm, mask)
    b = g.moe_gate(logits, topk, renormalize=renorm, loss_coef=0.05, token_mask=mask)
    assert all(torch.equal(p, q) for p, q in zip(a, b))  # the same bits again


# more tokens than the GPU's warps take at once, ragged at the end
@pytest.mark.parametrize("T,E,topk", [(5001, 256, 8), (6007, 130, 32), (9999, 100, 3), (20011, 64, 6), (39001, 32, 32),
                                      (78003, 16, 4), (156007, 8, 2), (160001, 3, 1), (3001, 300, 8), (2003, 700, 5)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_gate_many_tokens(T, E, topk, xd):
    logits = _draw((T, E), xd, T, 1.5)
    mask = torch.arange(T, device="cuda") % 5 != 1
    a = _check_gate(logits, topk, True, mask)
    b = g.moe_gate(logits, topk, renormalize=True, loss_coef=0.05, token_mask=mask)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("E", [5, 8, 32, 64, 200])
def test_gate_ties_and_ruled_out_experts(E):
    T = 12
    logits = _draw((T, E), "f32", E)
    logits[0] = 0.25                       # all equal: 0, 1, 2
    logits[1] = -0.0
    logits[1, 1::2] = 0.0                  # equal zeros of both signs
    logits[2] = float("-inf")              # nothing left
    logits[3] = float("-inf")
    logits[3, E - 1] = 2.0                 # fewer left than topk
    logits[4] = -3.0e38
    logits[4, 2] = -2.9e38                 # the type's lowest values
    logits[5, :] = torch.finfo(torch.float32).min
    logits[6, 0] = float("-inf")
    for renorm in (True, False):
        ids, w, *_ = _check_gate(logits[[0, 1, 2, 3, 6, 7, 8]].contiguous(), 3, renorm, None)
        assert ids[0].tolist() == [0, 1, 2] and ids[1].tolist() == [0, 1, 2]
        assert ids[2].tolist() == [0, 1, 2] and not w[2].any()
        assert ids[3].tolist() == [E - 1, 0, 1] and w[3, 1:].tolist() == [0.0, 0.0]
        ids, w, counts, loss = g.moe_gate(logits[4:6].contiguous(), 3, renormalize=renorm)
        assert ids.tolist() == [[2, 0, 1], [0, 1, 2]]
        assert w[0].tolist() == [1.0, 0.0, 0.0]
        assert torch.allclose(w[1], torch.full((3,), 1 / 3 if renorm else 1 / E, device="cuda"), rtol=1e-6, atol=0.0)


@pytest.mark.parametrize("E,topk", [(8, 2), (64, 4), (130, 3)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_gate_masked_tokens_may_hold_anything(E, topk, xd):
    T = 70
    logits = _draw((T, E), xd, 3)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[5] = mask[6] = mask[69] = mask[64] = 0
    clean = g.moe_gate(logits, topk, token_mask=mask)
    dw = torch.randn((T, topk), generator=_gen(1), device="cuda")
    dl = g.moe_gate_backward(logits, clean[0], clean[2], dw, torch.ones(1, device="cuda"), token_mask=mask)
    bad = logits.clone()
    bad[5], bad[6, 1], bad[69], bad[64] = float("nan"), float("inf"), float("inf"), float("-inf")
    ids, w, counts, loss = g.moe_gate(bad, topk, token_mask=mask)
    assert torch.equal(counts, clean[2]) and torch.equal(loss, clean[3])
    real = mask.bool()
    assert torch.equal(ids[real], clean[0][real]) and torch.equal(w, clean[1]) and not w[~real].any()
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    for row in ids.tolist():
        assert len(set(row)) == topk
    dwb = dw.clone()
    dwb[5] = float("nan")
    dlb = g.moe_gate_backward(bad, ids, counts, dwb, torch.ones(1, device="cuda"), token_mask=mask)
    assert torch.equal(dlb, dl) and not dlb[~real].any()


def test_gate_nan_stays_in_its_row():
    logits = _draw((40, 64), "f32", 4)
    logits[7, 3] = float("nan")
    ids, w, counts, loss = g.moe_gate(logits, 4)
    assert bool(torch.isnan(w[7]).all()) and ids[7, 0] == 3 and len(set(ids[7].tolist())) == 4
    assert not torch.isnan(w[torch.arange(40) != 7]).any()


@pytest.mark.parametrize("T,E", [(0, 8), (6, 8), (200, 300)])
def test_gate_no_tokens_or_all_masked(T, E):
    logits = _draw((T, E), "f32", 5)
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    ids, w, counts, loss = g.moe_gate(logits, 2, token_mask=mask)
    assert not w.any() and not counts.any() and loss.tolist() == [0.0]
    dl = g.moe_gate_backward(logits, ids, counts, torch.ones_like(w), torch.ones(1, device="cuda"), token_mask=mask)
    assert not dl.any()


@pytest.mark.parametrize("E,pad,offset", [(8, 8, 0), (8, 3, 1), (64, 1, 0), (256, 0, 1), (30, 2, 5), (128, 8, 8)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_gate_strides_and_alignment(E, pad, offset, xd):
    T = 37
    logits, _ = _strided((T, E), xd, pad, offset, 6)
    want = g.moe_gate(logits.contiguous(), 2)
    got = g.moe_gate(logits, 2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _check_gate(logits, 2, True, None)
    out, buf = _strided((T, E), xd, pad, offset)
    dw = torch.randn((T, 2), generator=_gen(2), device="cuda")
    g.fp8g_moe_gate_backward(logits, got[0], got[2], dw, None, out)
    assert torch.equal(out, g.moe_gate_backward(logits.contiguous(), got[0], got[2], dw))
    assert int(torch.isnan(buf).sum()) == buf.numel() - T * E
    inplace = logits.contiguous().clone()
    g.fp8g_moe_gate_backward(inplace, got[0], got[2], dw, None, inplace)
    assert torch.equal(inplace, out)


def test_gate_ids_out_of_range_have_no_gradient():
    logits = _draw((9, 16), "f32", 7)
    ids, w, counts, _ = g.moe_gate(logits, 2, renormalize=False)
    dw = torch.ones_like(w)
    cut = dw.clone()
    cut[4, 1] = cut[5, 0] = 0.0
    want = g.moe_gate_backward(logits, ids, counts, cut, renormalize=False)
    ids[4, 1], ids[5, 0] = -1, 16
    assert torch.equal(g.moe_gate_backward(logits, ids, counts, dw, renormalize=False), want)


# ------------------------------------------------------------------ combine

def _rows_of(T, topk, E, drop, seed):
    """The routed layout of random choices: entry_row [T, topk], row_token [M] (one dropped entry in `drop`)."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)]) if T else np.zeros((0, topk), np.int64)
    if drop:
        ids[rng.random(ids.shape) < 1.0 / drop] = -1
    entry = np.full((T, topk), -1, np.int32)
    tokens = []
    for e in range(E):
        for t, j in zip(*np.nonzero(ids == e)):
            entry[t, j] = len(tokens)
            tokens.append(t)
        tokens += [-1] * (-len(tokens) % 128)
    tokens += [-1] * 128
    return entry, np.array(tokens, np.int32)


@pytest.mark.parametrize("T,topk,E,N", [(1, 1, 1, 8), (2, 2, 4, 16), (5, 3, 4, 24), (64, 8, 32, 256), (37, 2, 8, 1000),
                                        (9, 12, 16, 136), (40, 4, 8, 4096), (3, 5, 6, 7168), (300, 2, 3, 64),
                                        (7, 2, 4, 16400)])
@pytest.mark.parametrize("yd", ["bf16", "f32"])
@pytest.mark.parametrize("drop,residual,weighted", [(0, False, True), (5, True, True), (5, True, False)])
def test_combine_and_gradient(T, topk, E, N, yd, drop, residual, weighted):
    entry, tokens = _rows_of(T, topk, E, drop, T + N)
    M = len(tokens)
    D = _draw((M, N), "bf16", 1)
    D[torch.from_numpy(tokens < 0).cuda()] = float("nan")  # padding rows are never read
    w = torch.rand((T, topk), generator=_gen(2), device="cuda") if weighted else None
    res = _draw((T, N), yd, 3) if residual else None
    er, rt = torch.from_numpy(entry).cuda(), torch.from_numpy(tokens).cuda()
    out = g.moe_combine(D, er, w, residual=res, out_dtype=DT[yd])
    Dn = np.nan_to_num(_np(D))
    wn = None if w is None else _np(w)
    want = ob.moe_combine(Dn, entry, wn, None if res is None else _np(res))
    size = ob.moe_combine(np.abs(Dn), entry, wn, None if res is None else np.abs(_np(res)))
    _within(out, want, (topk + 2) * U * size, yd, "out")
    dout = _draw((T, N), yd, 4)
    dD, dw = g.moe_combine_backward(dout, D, er, rt, w)
    rdD, rdw = ob.moe_combine_backward(_np(dout), Dn, entry, wn)
    _within(dD, rdD, 2 * U * np.abs(rdD), "bf16", "dD")
    assert not dD[rt < 0].any()
    if weighted:
        sdw = ob.moe_combine_backward(np.abs(_np(dout)), np.abs(Dn), entry, wn)[1]
        _within(dw, rdw, (N / 32 + 16) * U * sdw, "f32", "dweights")
        assert not dw[er < 0].any()
        again = g.moe_combine_backward(dout, D, er, rt, w)
        assert torch.equal(again[0], dD) and torch.equal(again[1], dw)
    else:
        assert dw is None
        full = torch.empty((T, topk), device="cuda")  # the weights' gradient is there for the asking
        g.fp8g_moe_combine_backward(dout, D, er, rt, None, torch.empty_like(dD), full)
        sdw = ob.moe_combine_backward(np.abs(_np(dout)), np.abs(Dn), entry)[1]
        _within(full, rdw, (N / 32 + 16) * U * sdw, "f32", "dweights")
    check_status()


@pytest.mark.parametrize("N,pad,offset", [(64, 8, 8), (1000, 24, 0), (4096, 8, 16)])
def test_combine_strides_and_in_place(N, pad, offset):
    T, topk, E = 21, 2, 4
    entry, tokens = _rows_of(T, topk, E, 6, 1)
    er, rt = torch.from_numpy(entry).cuda(), torch.from_numpy(tokens).cuda()
    D, _ = _strided((len(tokens), N), "bf16", pad, offset, 2)
    w = torch.rand((T, topk), generator=_gen(3), device="cuda")
    x, xbuf = _strided((T, N), "f32", pad, offset, 4)
    want = g.moe_combine(D.contiguous(), er, w, residual=x.contiguous())
    g.fp8g_moe_combine(D, er, w, x, residual=x)  # into the residual stream itself
    assert torch.equal(x, want) and int(torch.isnan(xbuf).sum()) == xbuf.numel() - T * N
    dout, _ = _strided((T, N), "bf16", pad, offset, 5)
    dD, dbuf = _strided((len(tokens), N), "bf16", pad, offset)
    dw = torch.empty((T, topk), device="cuda")
    g.fp8g_moe_combine_backward(dout, D, er, rt, w, dD, dw)
    rD, rw = g.moe_combine_backward(dout.contiguous(), D.contiguous(), er, rt, w)
    assert torch.equal(dD, rD) and torch.equal(dw, rw)
    assert int(torch.isnan(dbuf).sum()) == dbuf.numel() - len(tokens) * N


def test_combine_rows_out_of_range_are_left_out_and_reported():
    D = _draw((128, 64), "bf16", 6)
    er = torch.tensor([[0, 128], [2 ** 31 - 1, 5], [-7, -1]], dtype=torch.int32, device="cuda")
    out = g.moe_combine(D, er, None)
    assert g.fp8g_get_status() == 6
    assert torch.equal(out[0], D[0]) and torch.equal(out[1], D[5]) and not out[2].any()
    rt = torch.full((128,), -1, dtype=torch.int32, device="cuda")
    rt[0], rt[5] = 0, 1
    dout = _draw((3, 64), "bf16", 7)
    dD, dw = g.moe_combine_backward(dout, D, er, rt, torch.ones((3, 2), device="cuda"))
    assert g.fp8g_get_status() == 6
    assert torch.equal(dD[0], dout[0]) and torch.equal(dD[5], dout[1]) and not dD[1:5].any()
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and not dw[2].any()


def test_combine_no_tokens_and_no_rows():
    D = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert g.moe_combine(D, none).shape == (0, 64)
    er = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    assert not g.moe_combine(D, er).any()  # every entry dropped
    big = torch.full((256, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    rt = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    dD, dw = g.moe_combine_backward(torch.empty((0, 64), device="cuda"), big, none, rt,
                                    torch.empty((0, 2), device="cuda"))
    assert dD.shape == (256, 64) and not dD.any() and dw.numel() == 0


def test_combine_follows_the_routed_layout():
    # the layout that the library itself builds: identity experts bring every token back
    T, E, topk, K = 200, 8, 2, 256
    x = _draw((T, K), "bf16", 8)
    ids = g.moe_gate(_draw((T, E), "f32", 9), topk)[0]
    _, _, _, row_token, entry_row = g.route_gather_quantize_1x128(x, ids, E)
    D = torch.zeros((row_token.numel(), K), dtype=torch.bfloat16, device="cuda")
    D[row_token >= 0] = x[row_token[row_token >= 0].long()]
    w = torch.full((T, topk), 0.5, device="cuda")
    assert torch.equal(g.moe_combine(D, entry_row, w), x)
    dD, _ = g.moe_combine_backward(x, D, entry_row, row_token, torch.ones_like(w))
    assert torch.equal(dD, D)


# ------------------------------------------------------------------ gradient norm

def _clip_check(grads, max_norm, out=None):
    ng = [_np(t) for t in grads]
    n = sum(t.numel() for t in grads)
    k = (n / (256 * min(608, max(1, n // 8192))) + 40) * U  # squares a thread adds one after another
    rnorm, rout = ob.clip_grad_norm(ng, max_norm)
    lst = g.GradList(grads, out)
    got = g.grad_norm(lst)
    assert got.shape == (1,)
    assert abs(float(got) - rnorm) <= k * rnorm
    norm = g.clip_grad_norm(lst, max_norm)
    assert torch.equal(norm, got)
    for t, r in zip(lst.out, rout):
        _within(t, r, 2 * k * np.abs(r), "bf16" if t.dtype == torch.bfloat16 else "f32", "clipped")


@pytest.mark.parametrize("sizes", [(1,), (7, 1), (8,), (255, 256, 257), (8192,), (8193, 3), (1, 100000, 5, 70001),
                                   (0, 5, 0), (1200000,)])
@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("bf16", "f32")])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip(sizes, dtypes, in_place):
    grads = [_draw((n,), dtypes[i % len(dtypes)], i, 0.1) for i, n in enumerate(sizes)]
    _clip_check(grads, 0.05, None if in_place else [torch.empty_like(t) for t in grads])


@pytest.mark.parametrize("offset,out_offset", [(1, 1), (1, 0), (3, 2), (5, 5), (4, 4)])
@pytest.mark.parametrize("d", ["f32", "bf16"])
def test_clip_unaligned_views(offset, out_offset, d):
    n = 30011
    flat, oflat = _draw((n + 64,), d, 1), torch.full((n + 64,), float("nan"), dtype=DT[d], device="cuda")
    grads = [flat[offset: offset + 9], flat[offset + 20: offset + n]]
    out = [oflat[out_offset: out_offset + 9], oflat[out_offset + 20: out_offset + n]]
    _clip_check(grads, 1.0, out)
    assert int(torch.isnan(oflat).sum()) == oflat.numel() - (n - 11)


@pytest.mark.parametrize("count", [63, 64, 65, 1023, 1024, 1025, 2500])
def test_clip_many_tensors(count):
    flat = _draw((count * 37,), "f32", 2)
    grads = [flat[37 * i: 37 * i + 1 + i % 37] for i in range(count)]
    _clip_check(grads, 3.0, [torch.empty_like(t) for t in grads])


def test_clip_below_the_limit_changes_nothing():
    grads = [_draw((1000,), "bf16", 1, 1e-3), _draw((77,), "f32", 2, 1e-3)]
    keep = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads]
    g.clip_grad_norm(g.GradList(grads, out), 1.0)
    g.clip_grad_norm(grads, 1.0)
    assert all(torch.equal(a, b) for a, b in zip(grads + out, keep + keep))


def test_clip_zeros_and_values_that_are_not_finite():
    z = [torch.zeros(100, device="cuda"), torch.zeros(3, dtype=torch.bfloat16, device="cuda")]
    assert float(g.clip_grad_norm(z, 0.0, eps=0.0)) == 0.0 and not z[0].any()
    t = [torch.ones(50, device="cuda"), torch.ones(20000, device="cuda")]
    t[1][777] = float("inf")
    assert float(g.clip_grad_norm(t, 1.0)) == float("inf")
    assert not t[0].any() and bool(torch.isnan(t[1][777]))  # 1 * 0 and inf * 0
    t = [torch.ones(50, device="cuda"), torch.ones(20000, device="cuda")]
    t[1][0] = float("nan")
    assert bool(torch.isnan(g.clip_grad_norm(t, 1.0))) and bool(torch.isnan(t[0]).all())


# ------------------------------------------------------------------ streams, graphs, addresses past 32 bits

def _one_pass():
    """Every operator once on fixed inputs; the results as a list."""
    x, w = _draw((70, 1024), "bf16", 1), _draw((1024,), "bf16", 2)
    dy = _draw((70, 1024), "bf16", 3)
    logits = _draw((70, 64), "f32", 4)
    entry, tokens = _rows_of(70, 2, 8, 0, 5)
    er, rt = torch.from_numpy(entry).cuda(), torch.from_numpy(tokens).cuda()
    D = _draw((len(tokens), 1024), "bf16", 6)
    grads = [_draw((50000,), "f32", 7), _draw((333,), "bf16", 8)]
    outs = [torch.empty_like(t) for t in grads]
    lst = g.GradList(grads, outs)
    torch.cuda.synchronize()

    def step():
        y, mean, rstd = g.layer_norm(x, w)
        dx, dw, db = g.layer_norm_backward(dy, x, w, mean, rstd)
        ids, p, counts, loss = g.moe_gate(logits, 2)
        dl = g.moe_gate_backward(logits, ids, counts, p, loss)
        out = g.moe_combine(D, er, p, residual=y)
        dD, dp = g.moe_combine_backward(dy, D, er, rt, p)
        norm = g.clip_grad_norm(lst, 1.0)
        return [y, mean, rstd, dx, dw, db, ids, p, counts, loss, dl, out, dD, dp, norm, *outs]

    return step


def test_other_streams_and_graphs_give_the_same_bits():
    step = _one_pass()
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(4):
            busy = busy @ busy * 1e-3
        got = [t.clone() for t in step()]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    check_status()


def test_offsets_past_32_bits():
    # more than 2^31 elements from the first row to the last
    M, N = 131201, 16384
    x = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    x[-3:] = _draw((3, N), "bf16", 1)
    y = torch.empty_like(x)
    g.fp8g_layer_norm(x, None, None, y)
    assert torch.equal(y[-3:], g.layer_norm(x[-3:].clone())[0]) and not y[:2].any()
    er = torch.tensor([[M - 1, M - 2], [0, M - 3]], dtype=torch.int32, device="cuda")
    w = torch.rand((2, 2), generator=_gen(2), device="cuda")
    want = g.moe_combine(x[-3:].clone(), torch.tensor([[2, 1], [-1, 0]], dtype=torch.int32, device="cuda"), w)
    assert torch.equal(g.moe_combine(x, er, w), want)
    rt = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    rt[M - 1] = rt[M - 2] = 0
    rt[0] = rt[M - 3] = 1
    dout = _draw((2, N), "bf16", 3)
    y.fill_(1.0)
    dw = torch.empty((2, 2), device="cuda")
    g.fp8g_moe_combine_backward(dout, x, er, rt, w, y, dw)
    assert torch.equal(y[M - 1], (dout[0].float() * w[0, 0]).bfloat16()) and not y[1: M - 3].any()
    del y
    flat = x.view(-1)
    assert abs(float(g.grad_norm([flat])) - float(x[-3:].double().norm())) < 1e-4
    g.clip_grad_norm([flat], 1.0)
    assert abs(float(x[-3:].double().norm()) - 1.0) < 1e-2
    check_status()
