"""The whole-block training operators on the GPU against the 64-bit oracle: every type, odd and one-element sizes,
strides, unaligned tensors, masks that leave nothing, infinities and NaN in masked places, other streams and graphs.

Tolerances are error bounds of the formulas.  With u = 2^-24 (one fp32 rounding), a sum of n terms in which
each thread adds L of them one after another and the threads' sums join in a tree is off by at most (L + 12) u times
the sum of the terms' magnitudes; each further operation adds u.  A bf16 result adds its own rounding, 2^-8 of its
value at most (half a unit in the last of 8 bits, and as much again where the fp32 value crosses a midpoint).
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import e4m3_decode
from oracle import train_ops as ot
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import DT, U, _draw, _gen, _np, _strided, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _replayed(call, refill):
    """`call` captured once (after an eager call) and replayed on inputs that refill() changes."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    refill()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    return got


# ------------------------------------------------------------------ router

def _route_bounds(logits, ids, score):
    """Relative errors of the chosen scores: the exponential's argument (a difference, for a softmax) carries one rounding
    for each unit of it, exp and division 2 units in the last place (4 u) each; a softmax's sum adds 24 roundings and its
    terms' own errors, the mean of their distances at most log E < 8."""
    l = _np(logits)
    sel = np.take_along_axis(l, ids, 1)
    if score == "sigmoid":
        return (16 + np.abs(np.where(np.isfinite(sel), sel, 0))) * U
    mx = l.max(1, keepdims=True)
    d = np.where(np.isfinite(sel), mx - sel, 0)
    return (64 + d) * U


def _check_route(logits, k, bias=None, mask=None, **kw):
    ids, w, counts = g.moe_route(logits, k, bias=bias, token_mask=mask, **kw)
    check_status()
    rids, rw, rc = ot.moe_route(_np(logits), k, None if bias is None else _np(bias),
                                token_mask=None if mask is None else _np(mask), **kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.array_equal(counts.cpu().numpy(), rc)
    rel = _route_bounds(logits, rids, kw.get("score", "sigmoid"))
    _within(w, rw, 2 * (rel + rel.max(1, keepdims=True) + 40 * U) * np.abs(rw), "f32", "weights")
    return ids, w, counts


ROUTE_SIZES = [(1, 1, 1, 1, 1), (1, 4, 1, 1, 4), (3, 8, 2, 1, 3), (64, 256, 8, 4, 8), (65, 256, 1, 1, 8), (33, 64, 8, 8, 6),
               (40, 160, 8, 3, 6), (129, 128, 4, 2, 1), (31, 60, 12, 5, 7), (17, 96, 32, 9, 8), (2, 2048, 32, 4, 32),
               (5, 2048, 1, 1, 8), (9, 2016, 9, 2, 8), (700, 32, 32, 10, 10), (1000, 5, 5, 5, 5), (300, 24, 3, 2, 16),
               (4097, 256, 8, 4, 8), (5000, 40, 5, 2, 4), (50, 512, 16, 4, 8), (7, 1024, 2, 1, 4)]


@pytest.mark.parametrize("T,E,groups,kept,k", ROUTE_SIZES)
@pytest.mark.parametrize("dtype,score,biased,renorm", [
    ("f32", "sigmoid", True, True), ("bf16", "sigmoid", True, False), ("f32", "softmax", True, True),
    ("bf16", "softmax", False, True), ("f32", "sigmoid", False, False), ("bf16", "sigmoid", False, True)])
def test_route(T, E, groups, kept, k, dtype, score, biased, renorm):
    logits = _draw((T, E), dtype, 1, 1.0)
    bias = _draw((E,), "f32", 2, 0.1 if score == "sigmoid" else 0.3 / E) if biased else None
    mask = torch.rand(T, generator=_gen(3), device="cuda") < 0.8 if T % 2 else None
    _check_route(logits, k, bias, mask, score=score, groups=groups, topk_groups=kept, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,kept,k", [(256, 8, 4, 8), (256, 1, 1, 8), (64, 4, 2, 6), (160, 8, 3, 6)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_scores_that_lie_near_one_another(E, groups, kept, k, score):
    """Logits a few fp32 steps apart, biases that undo their differences but for less than fp32 tells apart, equal logits
    with a bias of zeros, saturated sigmoids: the choice is that of 64 bits."""
    T = 300
    base = torch.randn((T, 1), generator=_gen(5), device="cuda")
    near = base * (1 + torch.randint(0, 5, (T, E), generator=_gen(6), device="cuda") * 2.0 ** -23)
    zero = torch.zeros(E, device="cuda")
    kw = dict(score=score, groups=groups, topk_groups=kept)
    _check_route(near, k, zero, **kw)
    _check_route(near, k, None, **kw)
    l = torch.randn((T, E), generator=_gen(7), device="cuda")
    level = torch.sigmoid(l[0]) if score == "sigmoid" else torch.softmax(l[0], 0)
    _check_route(l[:1].expand(T, E).contiguous(), k, 0.5 - level, **kw)  # every choice score is about 1/2
    few = _draw((T, E), "bf16", 8).mul_(2).round_().div_(2)
    _check_route(few, k, zero, **kw)
    _check_route(few, k, None, **kw)
    _check_route(few, k, _draw((E,), "f32", 9, 1e-7), **kw)
    _check_route(l * 4 + 18, k, zero, **kw)
    _check_route(l * 4 - 18, k, zero, **kw)
    _check_route(l, k, _draw((E,), "f32", 10, 3.0) + 100.0, **kw)  # biases far above the scores


def test_route_ruled_out_experts():
    inf, T, E = float("inf"), 60, 64
    l = torch.randn((T, E), generator=_gen(1), device="cuda")
    out = torch.rand((T, E), generator=_gen(2), device="cuda") < 0.6
    out[3] = True                # nothing is left
    out[4, 1:] = True            # one
    out[5, :48] = True           # one group
    out[6] = False
    l[out] = -inf
    bias = _draw((E,), "f32", 3, 0.1)
    bias[7], bias[20:33] = -inf, -inf
    mask = torch.arange(T, device="cuda") != 9
    for b in (bias, None):
        for score in ("sigmoid", "softmax"):
            for groups, kept, k in ((1, 1, 6), (8, 3, 8), (4, 1, 12), (32, 20, 8)):
                _check_route(l, k, b, mask, score=score, groups=groups, topk_groups=kept)
    _check_route(l.bfloat16(), 8, None, mask, groups=8, topk_groups=4)
    _check_route(l.bfloat16(), 8, bias, mask, groups=8, topk_groups=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_not_a_number(dtype):
    """A NaN ranks first, its weight is NaN; other rows do not feel it."""
    l = _draw((40, 64), dtype, 1)
    l[5, 17] = float("nan")
    l[6, 40] = float("inf")
    for bias in (None, torch.zeros(64, device="cuda")):
        for groups, kept in ((1, 1), (8, 4)):
            ids, w, _ = g.moe_route(l, 4, bias=bias, groups=groups, topk_groups=kept, renormalize=False)
            rids, rw, _ = ot.moe_route(_np(l), 4, None if bias is None else _np(bias), groups=groups, topk_groups=kept,
                                       renormalize=False)
            assert np.array_equal(ids.cpu().numpy(), rids) and int(ids[5, 0]) == 17 and int(ids[6, 0]) == 40
            w = _np(w)
            assert np.isnan(w[5, 0]) and not np.isnan(w[5, 1:]).any() and w[6, 0] == 1.0
            rw[5, 0] = w[5, 0] = 0.0
            assert np.allclose(w, rw, rtol=1e-5, atol=0)


def test_route_strides_alignment_and_no_tokens():
    for dtype in ("f32", "bf16"):
        for pad, off in ((0, 1), (3, 0), (8, 0), (5, 3)):
            l, _ = _strided((50, 64), dtype, pad, off, seed=4)
            _check_route(l, 4, _draw((64,), "f32", 5, 0.1), groups=8, topk_groups=2)
            bias = _draw((65,), "f32", 6, 0.1)[1:]
            _check_route(l, 4, bias)
    ids, w, counts = g.moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2) and counts.tolist() == [0] * 8
    l = _draw((7, 8), "f32", 1)
    _check_route(l, 2, mask=torch.zeros(7, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("T,E,groups,kept,k", ROUTE_SIZES)
@pytest.mark.parametrize("dtype,score,renorm", [("f32", "sigmoid", True), ("bf16", "sigmoid", False),
                                                ("f32", "softmax", False), ("bf16", "softmax", True)])
def test_route_gradient(T, E, groups, kept, k, dtype, score, renorm):
    logits = _draw((T, E), dtype, 1)
    ids = torch.argsort(torch.rand((T, E), generator=_gen(2), device="cuda"), 1)[:, :k].to(torch.int32).contiguous()
    if k > 1 and T > 2:
        ids[1, 1] = ids[1, 0]  # the same expert twice
        ids[2, 0] = -1         # a dropped one
        ids[0, k - 1] = E
    dw = _draw((T, k), "f32", 3)
    mask = torch.rand(T, generator=_gen(4), device="cuda") < 0.8 if T % 2 else None
    got = g.moe_route_backward(logits, ids, dw, score=score, renormalize=renorm, scale=2.5, token_mask=mask)
    args = (_np(logits), ids.cpu().numpy())
    kw = dict(score=score, renormalize=renorm, scale=2.5, token_mask=None if mask is None else _np(mask))
    want = ot.moe_route_backward(*args, _np(dw), **kw)
    # The gradient's terms with all signs alike: each is off by at most 128 u of itself (scores 64 + distance, the inner
    # sum's 40, a few more); what cancels between them does not cancel in the error.
    s = ot.route_scores(args[0], score)
    at = np.clip(args[1], 0, E - 1)
    inside = (args[1] >= 0) & (args[1] < E)
    d = np.where(inside, np.abs(_np(dw)) * 2.5, 0)
    sel = np.where(inside, np.take_along_axis(s, at, 1), 0)
    if renorm:
        total = np.maximum(sel.sum(1, keepdims=True), 1e-300)
        d = np.where(inside, (d + (d * sel).sum(1, keepdims=True) / total) / total, 0)
    G = np.zeros((T, E))
    np.add.at(G, (np.arange(T)[:, None], at), d)
    size = G * s * (1 - s) if score == "sigmoid" else s * (G + (G * s).sum(1, keepdims=True))
    far = np.abs(args[0]) if score == "sigmoid" else args[0].max(1, keepdims=True) - args[0]
    _within(got, want, (160 + far + far.max()) * U * size, dtype, "dlogits")
    again = logits.clone()  # in place
    g.fp8g_moe_route_backward(again, ids, dw, again, score=score, renormalize=renorm, scale=2.5, token_mask=mask)
    assert torch.equal(again, got)


def test_route_gradient_strides_and_masked_places():
    l, _ = _strided((30, 33), "f32", 5, 3, seed=1)
    out, buf = _strided((30, 33), "f32", 2, 1)
    l[4] = float("nan")
    l[5, 3] = float("-inf")
    ids = torch.randint(0, 33, (30, 4), generator=_gen(2), device="cuda", dtype=torch.int32)
    ids[5, 0] = 3
    mask = torch.arange(30, device="cuda") != 4
    for score in ("sigmoid", "softmax"):
        g.fp8g_moe_route_backward(l, ids, _draw((30, 4), "f32", 3), out, score=score, token_mask=mask)
        assert torch.equal(out[4], torch.zeros(33, device="cuda")) and torch.isfinite(out).all() and out[5, 3] == 0
        assert torch.isnan(buf[:1]).all() and torch.isnan(buf[1:1 + 30 * 35].view(30, 35)[:, 33:]).all()
    assert g.moe_route_backward(l[:0], ids[:0], _draw((0, 4), "f32", 3)).shape == (0, 33)


def test_route_in_a_graph_and_on_another_stream():
    l = _draw((3000, 64), "f32", 1)
    other = _draw((3000, 64), "f32", 2)
    bias = _draw((64,), "f32", 3, 0.1)
    kw = dict(bias=bias, groups=8, topk_groups=4)
    got = _replayed(lambda: g.moe_route(l, 6, **kw), lambda: l.copy_(other))
    want = g.moe_route(other, 6, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = g.moe_route(other, 6, **kw)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


# ------------------------------------------------------------------ norms around a block

def _rms(a):
    return np.sqrt((a * a).mean(1, keepdims=True))


def _check_norm(x, f, w, gate, scale, post, pw, got, yd):
    h, y, rstd, rstd_f = got
    xn, fn, wn, gn, pn = (None if t is None else _np(t) for t in (x, f, w, gate, pw))
    rh, ry, rr, rrf = ot.residual_rms_norm(xn, fn, wn, gn, scale, post, pn)
    N = xn.shape[1]
    k = (N / 512 + 64) * U  # a sum's, and so at least twice a root's relative error
    dh = np.zeros_like(rh)
    if f is not None:
        dh = 2 * k * np.abs(rh - xn) + 4 * U * (np.abs(rh) + np.abs(xn))
        _within(h, rh, dh, {v: n for n, v in DT.items()}[x.dtype], "h")
    if post:
        _within(rstd_f, rrf, k * rrf, "f32", "rstd_f")
    moved = (_rms(dh) / np.maximum(_rms(rh), 1e-30))[:, 0]  # how far h's errors move the root, relatively
    _within(rstd, rr, (k + moved) * rr, "f32", "rstd")
    wa = np.ones(N) if wn is None else np.abs(wn)
    _within(y, ry, (dh + np.abs(rh) * (2 * k + moved[:, None])) * rr[:, None] * wa * 1.01, yd, "y")
    return rr, rrf


def _check_norm_grad(dy, dh, h, f, rstd, rstd_f, w, gate, scale, post, pw, got, sd, bd):
    arrays = [None if t is None else _np(t) for t in (dy, dh, h, f, rstd, rstd_f)]
    wn, gn, pn = (None if t is None else _np(t) for t in (w, gate, pw))
    want = ot.residual_rms_norm_backward(*arrays, wn, gn, scale, post, pn)
    dyn, dhn, hn, fn, r, rf = arrays
    M, N = want[0].shape
    k = (N / 512 + 64) * U
    rows = (M / 64 + 100) * U
    err = np.zeros((M, N)) if dhn is None else 2 * U * np.abs(dhn)
    if dyn is not None:
        e, gw = np.abs(hn) * r[:, None], np.abs(dyn) * (1.0 if wn is None else np.abs(wn))
        err = err + r[:, None] * (8 * U * gw + e * (k + 8 * U) * (gw * e).mean(1, keepdims=True)) + 2 * U * np.abs(want[0])
        if got[2] is not None:
            _within(got[2], want[2], 2 * rows * (np.abs(dyn) * e).sum(0), "f32", "dweight")
    _within(got[0], want[0], err, sd, "dx")
    if fn is None:
        return
    a = abs(scale) * (1.0 if gn is None else np.abs(gn)) * (1.0 if pn is None else np.abs(pn))
    q = np.abs(want[0]) * a
    ferr = err * a + 8 * U * q
    kf = np.abs(fn)
    if post:
        kf = kf * rf[:, None]
        ferr = rf[:, None] * (ferr + kf * ((err * a * kf).mean(1, keepdims=True) + (k + 8 * U) * (q * kf).mean(1, keepdims=True))
                              + 4 * U * q)
    _within(got[1], want[1], ferr, bd, "df")
    S = abs(scale) * ((err + rows * np.abs(want[0])) * kf * 2).sum(0)
    if got[3] is not None:
        _within(got[3], want[3], S * (1.0 if pn is None else np.abs(pn)), "f32", "dgate")
    if got[4] is not None:
        _within(got[4], want[4], S * (1.0 if gn is None else np.abs(gn)), "f32", "dpost")


RES_SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 31), (3, 64), (70, 64), (7, 127), (130, 128), (3, 129), (9, 256), (9, 264),
             (40, 512), (2, 520), (2, 1000), (33, 1024), (2, 1025), (3, 2048), (5, 4099), (4, 4096), (3, 7168), (161, 7168),
             (2, 8200), (700, 2048), (3, 16384), (2, 16392), (2, 20001), (1, 40000), (2000, 72), (400, 1032)]
RES_TYPES = [("bf16", "bf16", "bf16"), ("f32", "bf16", "f32"), ("f32", "f32", "f32"), ("bf16", "f32", "f32"),
             ("f32", "bf16", "bf16")]


@pytest.mark.parametrize("M,N", RES_SIZES)
@pytest.mark.parametrize("sd,bd,wd", RES_TYPES)
def test_residual_norm_and_gradients(M, N, sd, bd, wd):
    x, f = _draw((M, N), sd, 1, 2.0, 0.3), _draw((M, N), bd, 2, 0.7)
    w, pw, gate = _draw((N,), wd, 3, 0.3, 1.0), _draw((N,), wd, 4, 0.3, 1.0), _draw((N,), wd, 5, 0.3, 0.5)
    dy, dh = _draw((M, N), bd, 6, 0.02), _draw((M, N), sd, 7, 0.02)
    for post, gated in ((True, True), (False, False), (True, False), (False, True)):
        p, a = pw if post else None, gate if gated else None
        got = g.residual_rms_norm(x, f, w, gate=a, scale=0.75, post_norm=post, post_weight=p)
        _check_norm(x, f, w, a, 0.75, post, p, got, bd)
        h, _, rstd, rstd_f = got
        grads = g.residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, w, gate=a, scale=0.75, post_norm=post,
                                             post_weight=p)
        _check_norm_grad(dy, dh, h, f, rstd, rstd_f, w, a, 0.75, post, p, grads, sd, bd)
    check_status()


@pytest.mark.parametrize("M,N", [(3, 64), (37, 200), (5, 4099), (40, 7168), (2, 17000)])
@pytest.mark.parametrize("sd,bd", [("bf16", "bf16"), ("f32", "bf16")])
def test_residual_norm_parts(M, N, sd, bd):
    """The norm alone, the residual alone, without weights, and gradients that are not there."""
    x, f, w = _draw((M, N), sd, 1), _draw((M, N), bd, 2), _draw((N,), "f32", 3, 0.2, 1.0)
    dy, dh = _draw((M, N), bd, 4), _draw((M, N), sd, 5)
    h, y, rstd, rstd_f = g.residual_rms_norm(x, None, w, out_dtype=DT[bd])
    assert h is x and rstd_f is None
    _check_norm(x, None, w, None, 1.0, False, None, (h, y, rstd, rstd_f), bd)
    for d in (dh, None):
        got = g.residual_rms_norm_backward(dy, d, x, None, rstd, None, w)
        assert got[1] is None and got[3] is None and got[4] is None
        _check_norm_grad(dy, d, x, None, rstd, None, w, None, 1.0, False, None, got, sd, bd)
    # no weights at all, no gradients of weights
    h, y, rstd, rstd_f = g.residual_rms_norm(x, f, scale=-0.5, post_norm=True)
    _check_norm(x, f, None, None, -0.5, True, None, (h, y, rstd, rstd_f), bd)
    got = g.residual_rms_norm_backward(dy, None, h, f, rstd, rstd_f, scale=-0.5, post_norm=True)
    assert got[2:] == (None, None, None)
    _check_norm_grad(dy, None, h, f, rstd, rstd_f, None, None, -0.5, True, None, got, sd, bd)
    # the residual alone (a last block's), in place, and its gradient
    x2 = x.clone()
    g.fp8g_residual_rms_norm(x2, f, None, x2, None, gate=w, scale=0.5)
    want = _np(x) + 0.5 * _np(f) * _np(w)
    _within(x2, want, 4 * U * (np.abs(_np(x)) + np.abs(want)), sd, "h")
    d2, df, dg = dh.clone(), torch.empty_like(f), torch.empty(N, device="cuda")
    g.fp8g_residual_rms_norm_backward(None, d2, None, f, None, None, None, d2, df, dgate=dg, gate=w, scale=0.5)
    assert torch.equal(d2, dh)
    _check_norm_grad(None, dh, None, f, None, None, None, w, 0.5, False, None, (d2, df, None, dg, None), sd, bd)
    # f is not needed where no gate's gradient is
    df2 = torch.empty_like(f)
    g.fp8g_residual_rms_norm_backward(None, dh, None, None, None, None, None, torch.empty_like(dh), df2, gate=w, scale=0.5)
    assert torch.equal(df, df2)


@pytest.mark.parametrize("N", [63, 64, 520, 4096, 7168])
def test_residual_norm_strides_and_alignment(N):
    M = 37
    for sd, bd, wd in RES_TYPES[:3]:
        for pad, off in ((8, 0), (0, 1), (3, 0), (8, 8), (5, 2)):
            x, f = _strided((M, N), sd, pad, off, seed=1)[0], _strided((M, N), bd, pad + 8, off, seed=2)[0]
            h, hb = _strided((M, N), sd, pad, off)
            y, yb = _strided((M, N), bd, 8, off)
            w = _draw((N + 1,), wd, 3, 0.2, 1.0)[1:]
            pw, gate = _draw((N,), wd, 4, 0.2, 1.0), _draw((N + 3,), wd, 5, 0.2, 1.0)[3:]
            rstd, rstd_f = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
            g.fp8g_residual_rms_norm(x, f, w, h, y, rstd, rstd_f, gate, 0.5, True, pw)
            _check_norm(x, f, w, gate, 0.5, True, pw, (h, y, rstd, rstd_f), bd)
            for b, ld in ((hb, N + pad), (yb, N + 8)):  # nothing beside the rows was written
                assert torch.isnan(b[:off]).all() and torch.isnan(b[off + M * ld:]).all()
                assert torch.isnan(b[off: off + M * ld].view(M, ld)[:, N:]).all()
            dy, dh = _strided((M, N), bd, pad, off, seed=6)[0], _strided((M, N), sd, 8, off, seed=7)[0]
            dx, dxb = _strided((M, N), sd, pad, off)
            df, dfb = _strided((M, N), bd, 16, off)
            dw, dg, dp = (torch.empty(N, device="cuda") for _ in range(3))
            g.fp8g_residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, w, dx, df, dw, dg, dp, gate, 0.5, True, pw)
            _check_norm_grad(dy, dh, h, f, rstd, rstd_f, w, gate, 0.5, True, pw, (dx, df, dw, dg, dp), sd, bd)
            for b, ld in ((dxb, N + pad), (dfb, N + 16)):
                assert torch.isnan(b[:off]).all() and torch.isnan(b[off + M * ld:]).all()
                assert torch.isnan(b[off: off + M * ld].view(M, ld)[:, N:]).all()
    check_status()


def test_residual_norm_of_no_rows_and_of_zeros():
    z = torch.empty((0, 64), device="cuda")
    h, y, rstd, _ = g.residual_rms_norm(z, z, torch.ones(64, device="cuda"), gate=torch.ones(64, device="cuda"))
    assert h.shape == y.shape == (0, 64)
    got = g.residual_rms_norm_backward(z, z, z, z, rstd, None, torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    assert got[0].shape == (0, 64) and got[2].abs().sum() == 0 and got[3].abs().sum() == 0
    x = torch.zeros((3, 1000), device="cuda")
    h, y, rstd, rstd_f = g.residual_rms_norm(x, x, post_norm=True, eps=1e-6)
    assert h.abs().sum() == 0 and y.abs().sum() == 0 and torch.allclose(rstd, torch.full((3,), 1e3, device="cuda"))


def test_residual_norm_repeats_and_in_a_graph():
    """The same bits twice, and from a replayed graph with other inputs."""
    for M, N in ((900, 256), (300, 7168)):
        t = [_draw((M, N), "bf16", s) for s in range(4)]
        new = [_draw((M, N), "bf16", s) for s in range(4, 8)]
        w = _draw((N,), "f32", 9)

        def call():
            h, y, rstd, rstd_f = g.residual_rms_norm(t[0], t[1], w, gate=w, post_norm=True, post_weight=w)
            return (h, y, *g.residual_rms_norm_backward(t[2], t[3], h, t[1], rstd, rstd_f, w, w, 1.0, True, w))

        first, second = call(), call()
        assert all(torch.equal(a, b) for a, b in zip(first, second))
        got = _replayed(call, lambda: [a.copy_(b) for a, b in zip(t, new)])
        want = call()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ gated activation

def _glu_error(gu):
    """The relative error of fp32 h: e^-g carries a rounding for each unit of its exponent, a dozen more follow."""
    n = _np(gu)
    return (np.abs(n[..., : n.shape[-1] // 2]) + 16) * U


def _check_glu(gu, q, s, rows=None):
    """Codes within half a step of h / scale (2^-4 of itself, or 2^-10), with h's and the scale's errors, and scales."""
    h, rel = ot.swiglu(_np(gu)), _glu_error(gu)
    M, F = h.shape
    top = np.abs(h).reshape(M, F // 128, 128).max(2)
    worst = rel.reshape(M, F // 128, 128).max(2) + 8 * U
    got = _np(s)[:, :M].T
    assert np.all(np.abs(got - top / 448) <= worst * top / 448 + 1e-44)
    scale = np.repeat(top / 448, 128, axis=1)
    y = np.divide(h, scale, out=np.zeros_like(h), where=scale > 0)
    off = np.abs(e4m3_decode(q.cpu().numpy()) - y)
    slack = (rel + np.repeat(worst, 128, axis=1) + 8 * U) * np.abs(y)
    assert np.all(off <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + slack + 2.0 ** -30)


@pytest.mark.parametrize("M,F", [(1, 128), (3, 256), (7, 640), (130, 128), (33, 2048), (500, 4096), (5, 7168), (2, 16384)])
def test_swiglu_and_quantisation(M, F):
    gu = _draw((M, 2 * F), "bf16", 1, 2.0)
    gu[:, :128] *= 20  # saturated gates
    q, s, h = g.swiglu_quantize_1x128(gu, keep=True)
    check_status()
    _check_glu(gu, q, s)
    want = ot.swiglu(_np(gu))
    # s(g) below 2^-126 (g < -87), which fp32 instructions without subnormals make 0, takes up to 2^-126 |g u| with it
    lost = 2.0 ** -126 * np.abs(_np(gu)[:, :F] * _np(gu)[:, F:]) * (_np(gu)[:, :F] < -87)
    _within(h, want, _glu_error(gu) * np.abs(want) + lost, "bf16", "h")
    assert torch.equal(h, g.swiglu(gu))
    assert torch.equal(q, g.swiglu_quantize_1x128(gu)[0]) and g.swiglu_quantize_1x128(gu)[2] is None


@pytest.mark.parametrize("M,F", [(1, 8), (3, 24), (130, 136), (9, 1000), (400, 2048), (5, 7176)])
def test_swiglu_gradient(M, F):
    gu, dh = _draw((M, 2 * F), "bf16", 1, 2.0), _draw((M, F), "bf16", 2)
    dgu, h = g.swiglu_backward(dh, gu)
    assert torch.equal(h, g.swiglu(gu)) and g.swiglu_backward(dh, gu, keep=False)[1] is None
    n, d = _np(gu), _np(dh)
    gate, up = n[:, :F], n[:, F:]
    s, a = ot.route_scores(gate), np.abs(gate)
    rel = (a + 16) * U
    # 1 + g (1 - s) is off by |g| times (s rel + u) and a few roundings; s by rel
    bound = np.concatenate([np.abs(d * up) * s * (rel * (1 + a) * 2 + a * (s * rel + 4 * U)), np.abs(d * gate) * s * rel], 1)
    _within(dgu, ot.swiglu_backward(d, n), bound, "bf16", "dgu")
    again = gu.clone()
    g.fp8g_swiglu_backward(dh, again, again)
    assert torch.equal(again, dgu)


def test_swiglu_extremes():
    """Zeros, blocks whose scale is below 2^-126, and gates far out on both sides."""
    gu = torch.zeros((6, 512), dtype=torch.bfloat16, device="cuda")
    gu[1] = 1e-20
    gu[2, :256], gu[2, 256:] = 1.0, 2.0 ** -130  # h about 2^-130: fp32 has it to 2^-149
    gu[3, :256], gu[3, 256:] = -200.0, 3.0
    gu[4, :256], gu[4, 256:] = 200.0, 3.0
    gu[5, 0], gu[5, 256] = 5.0, 5.0
    q, s, h = g.swiglu_quantize_1x128(gu, keep=True)
    assert torch.isfinite(h).all() and torch.isfinite(s).all()
    v = e4m3_decode(q.cpu().numpy())
    assert not v[0].any() and not s[:, 0].any() and not v[5, 1:].any() and v[5, 0] == 448.0
    assert np.all(np.abs(v[2]) == 448.0)  # all alike, so all are the block's largest
    assert np.all(np.abs(h[3].float().cpu().numpy()) <= 1e-30) and torch.equal(h[4], torch.full_like(h[4], 600.0))
    dgu, _ = g.swiglu_backward(torch.ones((6, 256), dtype=torch.bfloat16, device="cuda"), gu)
    assert torch.isfinite(dgu).all()


def test_swiglu_strides():
    M, F = 21, 256
    for pad in (0, 8, 24):
        gu, _ = _strided((M, 2 * F), "bf16", pad, 8, seed=1)
        h, hb = _strided((M, F), "bf16", pad + 8, 16)
        qb = torch.full((M, F + 32), 0x7F, dtype=torch.uint8, device="cuda")
        s = torch.full((F // 128, 40), float("nan"), device="cuda")
        g.fp8_swiglu_quantize_1x128(gu, qb[:, :F], s, h)
        _check_glu(gu, qb[:, :F], s)
        assert (qb[:, F:] == 0x7F).all() and torch.isnan(s[:, M:]).all()
        assert torch.isnan(hb[16: 16 + M * (F + pad + 8)].view(M, -1)[:, F:]).all()
        dh, _ = _strided((M, F), "bf16", pad, 0, seed=2)
        dgu, db = _strided((M, 2 * F), "bf16", pad + 16, 8)
        g.fp8g_swiglu_backward(dh, gu, dgu)
        assert torch.equal(dgu, g.swiglu_backward(dh.contiguous(), gu.contiguous())[0])
        assert torch.isnan(db[8: 8 + M * (2 * F + pad + 16)].view(M, -1)[:, 2 * F:]).all()
    q, s, h = g.swiglu_quantize_1x128(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), keep=True)
    assert q.shape == h.shape == (0, 128)


@pytest.mark.parametrize("E,cap,F", [(1, 1, 128), (4, 5, 256), (32, 64, 2048), (7, 300, 384), (200, 3, 128)])
def test_swiglu_masked(E, cap, F):
    gu = _draw((E, cap, 2 * F), "bf16", 1, 2.0)
    counts = torch.randint(0, cap + 1, (E,), generator=_gen(2), device="cuda", dtype=torch.int32)
    counts[0] = cap
    if E > 3:
        counts[1], counts[2], counts[3] = 0, -3, cap + 9  # clamped
    full = gu.clone()
    valid = torch.arange(cap, device="cuda")[None] < counts[:, None].clamp(0, cap)
    full[~valid] = float("nan")  # what lies behind the counts is not read
    q = torch.full((E, cap, F), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((F // 128, (E * cap + 3) // 4 * 4), float("nan"), device="cuda")
    g.fp8_swiglu_quantize_1x128_masked(full, q, s, counts)
    check_status()
    wq, ws, _ = g.swiglu_quantize_1x128(gu.view(E * cap, 2 * F))
    v = valid.reshape(-1)
    assert torch.equal(q.view(E * cap, F)[v], wq[v]) and (q.view(E * cap, F)[~v] == 0x7F).all()
    assert torch.equal(s[:, : E * cap][:, v], ws[:, : E * cap][:, v]) and torch.isnan(s[:, : E * cap][:, ~v]).all()


# ------------------------------------------------------------------ AdamW

def _tensors(sizes, kinds, seed, std, flat):
    """Tensors of their own, or views into one flat buffer a type (few of them aligned)."""
    if not flat:
        return [_draw((n,), k, seed + i, std) for i, (n, k) in enumerate(zip(sizes, kinds))]
    bufs = {k: _draw((sum(n for n, kk in zip(sizes, kinds) if kk == k) + 3,), k, seed, std) for k in set(kinds)}
    at, out = {k: 1 for k in bufs}, []
    for n, k in zip(sizes, kinds):
        out.append(bufs[k][at[k]: at[k] + n])
        at[k] += n
    return out


def _check_adam(before, after, grads, t, lr, b1, b2, eps, wd, coef, bits, what):
    """before, after: (param, master or None, m, v, m_scale, v_scale) of one tensor."""
    p0 = _np(before[0] if before[1] is None else before[1]).reshape(-1)
    gr = _np(grads).reshape(-1)
    if bits == 32:
        m0, v0 = _np(before[2]), _np(before[3])
    else:
        m0 = ot.state_values(before[2].cpu().numpy(), before[4].cpu().numpy())
        root = ot.state_values(before[3].cpu().numpy(), before[5].cpu().numpy())
        v0 = root.astype(np.float64) ** 2
    p, m, v = ot.adamw(p0, gr, m0, v0, t, lr, b1, b2, eps, wd, coef)
    # m and v: two products and a sum, the gradient's factor and its own rounding
    em = 4 * U * (np.abs(b1 * m0) + 2 * np.abs((1 - b1) * gr * coef))
    ev = 4 * U * (b2 * v0 + 4 * (1 - b2) * (gr * coef) ** 2)
    c1, c2 = 1 - b1 ** t, 1 - b2 ** t
    den = np.sqrt(v / c2) + eps
    step = np.abs(m / c1 / den)
    ep = 2 * U * (np.abs(p) + np.abs(p0)) + lr * (em / c1 / den + step * (0.5 * ev / np.maximum(v, 1e-300) + 12 * U)
                                                + 4 * U * wd * np.abs(p0))
    kind = {torch.bfloat16: "bf16", torch.float32: "f32"}[after[0].dtype]
    if after[1] is not None:
        _within(after[1].reshape(-1), p, ep, "f32", what + " master")
        assert torch.equal(after[0].reshape(-1), after[1].bfloat16().reshape(-1))
    else:
        _within(after[0].reshape(-1), p, ep, kind, what + " param")
    if bits == 32:
        _within(after[2], m, em, "f32", what + " m")
        _within(after[3], v, ev, "f32", what + " v")
        return
    m32, r32 = ot.adamw_states(gr, m0, root, b1, b2, coef)
    for x, codes, scales, is_root in ((m32, after[2], after[4], False), (r32, after[3], after[5], True)):
        wc, wsc = ot.encode_states(x, t, is_root)
        assert np.array_equal(scales.cpu().numpy(), wsc), what
        assert np.array_equal(codes.cpu().numpy(), wc), what


ADAM_SIZES = [1, 7, 127, 128, 129, 1000, 2048, 2049, 5000, 40001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("pd,gd,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                          ("bf16", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True)])
def test_adamw(bits, flat, pd, gd, master):
    n = len(ADAM_SIZES)
    params, grads = _tensors(ADAM_SIZES, [pd] * n, 1, 0.1, flat), _tensors(ADAM_SIZES, [gd] * n, 50, 0.01, flat)
    decay = [0.1 * (i % 3) for i in range(n)]
    opt = g.AdamWList(params, grads, masters=master, state_bits=bits, weight_decay=decay)
    norm = torch.tensor([2.0], device="cuda")
    lr = torch.tensor([3e-3], device="cuda")
    for t in range(1, 4):
        rows = lambda: [tuple(None if x is None else x.clone() for x in r) for r in zip(  # noqa: E731
            opt.params, opt.masters, opt.m, opt.v, opt.m_scales, opt.v_scales)]
        before = rows()
        grads_now = [d.clone() for d in grads]
        clip = t == 2
        g.adamw_step(opt, lr if t == 3 else 3e-3, 0.9, 0.95, 1e-8, norm=norm if clip else None, max_norm=0.5, norm_eps=0.0)
        assert int(opt.step) == t
        for i, (a, b) in enumerate(zip(before, rows())):
            _check_adam(a, b, grads_now[i], t, float(np.float32(3e-3)) if t == 3 else 3e-3, 0.9, 0.95, 1e-8, decay[i],
                        0.25 if clip else 1.0, bits, f"tensor {i} step {t}")
        for i, d in enumerate(grads):
            d.copy_(_draw((ADAM_SIZES[i],), gd, 100 * t + i, 0.01 / t))
    check_status()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_tensors_and_large_ones(bits):
    """More tensors than a launch's table holds, empty ones among them, and one beyond 2^24 values."""
    sizes = [(i * 37) % 300 for i in range(900)] + [(1 << 24) + 5]
    kinds = ["f32" if i % 2 else "bf16" for i in range(len(sizes))]
    params = [_draw((n,), k, i, 0.1) for i, (n, k) in enumerate(zip(sizes, kinds))]
    grads = [_draw((n,), "f32", 2000 + i, 0.01) for i, n in enumerate(sizes)]
    before = [p.clone() for p in params]
    opt = g.AdamWList(params, grads, masters=True, state_bits=bits)
    g.adamw_step(opt, 1e-2)
    check_status()
    for i in list(range(0, 900, 53)) + [384, 385, 899, 900]:
        z, zs = torch.zeros_like(opt.m[i]), None if bits == 32 else torch.zeros_like(opt.m_scales[i])
        first = (before[i], before[i].float() if kinds[i] == "bf16" else None, z, z, zs, zs)
        _check_adam(first, (params[i], opt.masters[i], opt.m[i], opt.v[i], opt.m_scales[i], opt.v_scales[i]), grads[i], 1,
                    1e-2, 0.9, 0.999, 1e-8, float(np.float32(0.01)), 1.0, bits, f"tensor {i}")


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_leaves_a_step_out_where_the_norm_is_not_finite(bits):
    p, d = _draw((1000,), "f32", 1), _draw((1000,), "bf16", 2)
    opt = g.AdamWList([p], [d], state_bits=bits)
    g.adamw_step(opt, 1e-2)
    held = [t.clone() for t in (p, opt.m[0], opt.v[0], opt.step)]
    for bad in (float("nan"), float("inf")):
        g.adamw_step(opt, 1e-2, norm=torch.tensor([bad], device="cuda"), max_norm=1.0)
        assert all(torch.equal(a, b) for a, b in zip(held, (p, opt.m[0], opt.v[0], opt.step)))
    g.adamw_step(opt, 1e-2, norm=torch.tensor([1e-9], device="cuda"))  # without max_norm: taken as they are
    assert int(opt.step) == 2 and torch.isfinite(p).all()


def test_adamw_zero_and_tiny_gradients():
    """Blocks without gradients stay as they are but for the decay; states too small for a scale become 0."""
    p = torch.ones(384, device="cuda")
    d = torch.zeros(384, device="cuda")
    d[128:256] = 1e-25
    d[256:] = 1e-12
    opt = g.AdamWList([p], [d], state_bits=8, weight_decay=0.5)
    for _ in range(3):
        g.adamw_step(opt, 1e-3)
    assert torch.isfinite(p).all() and torch.allclose(p[:128], torch.full((128,), (1 - 5e-4) ** 3, device="cuda"))
    assert not opt.m[0][:256].any() and opt.m_scales[0][:2].tolist() == [0.0, 0.0] and opt.v[0][256:].all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_in_a_graph(bits):
    """Replays count the steps on, read the rate and the norm from the device, and give the eager bits."""
    sizes = [3000, 17, 129]

    def build():
        params, grads = _tensors(sizes, ["bf16"] * 3, 1, 0.1, False), _tensors(sizes, ["f32"] * 3, 9, 0.01, False)
        return g.AdamWList(params, grads, masters=True, state_bits=bits)

    lr = torch.tensor([1e-2], device="cuda")
    a, b = build(), build()
    norm = torch.tensor([4.0], device="cuda")
    call = lambda o: g.adamw_step(o, lr, norm=norm, max_norm=1.0)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(a)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    for i in range(3):
        lr.fill_(1e-2 / (i + 1))
        graph.replay()
    torch.cuda.synchronize()
    lr.fill_(1e-2)
    call(b)
    for i in range(3):
        lr.fill_(1e-2 / (i + 1))
        call(b)
    assert int(a.step) == int(b.step) == 4
    for x, y in zip(a.tensors, b.tensors):
        assert torch.equal(x, y)


def test_adamw_list_refuses_overlaps_and_tensors_that_moved():
    p, d = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    for params, grads in (([p, p], [d, d]), ([p[:40], p[32:]], [d[:40], d[32:]]), ([p], [p])):
        with pytest.raises(ValueError):
            g.AdamWList(params, grads)
    with pytest.raises(ValueError):
        g.AdamWList([p], [d], m=[torch.zeros(64, device="cuda")], v=[p])
    opt = g.AdamWList([p], [d])
    d.data = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        g.adamw_step(opt, 1e-3)


def test_adamw_goes_on_from_given_states():
    """Two steps by one list are those of a list each, the second with the first one's states."""
    for bits in (32, 8):
        p, d = _draw((777,), "f32", 1), _draw((777,), "f32", 2)
        q = p.clone()
        one = g.AdamWList([p], [d], state_bits=bits)
        g.adamw_step(one, 1e-2)
        g.adamw_step(one, 1e-2)
        first = g.AdamWList([q], [d], state_bits=bits)
        g.adamw_step(first, 1e-2)
        more = {} if bits == 32 else {"m_scales": first.m_scales, "v_scales": first.v_scales}
        m = first.m if bits == 32 else [first.m[0].view(torch.float8_e4m3fn)]
        second = g.AdamWList([q], [d], state_bits=bits, m=m, v=first.v, step=first.step, **more)
        g.adamw_step(second, 1e-2)
        assert torch.equal(p, q) and int(second.step) == 2
