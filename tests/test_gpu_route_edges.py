"""The router and its gradient where fp32 scores run out: chosen scores whose sum is below fp32's normal range, or below all
of it, and biases so large that a score hardly shows in its sum with them."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import train_ops as ot
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import U, _draw, _gen, _np, _within

pytestmark = pytest.mark.gpu

FORMS = [(16, 1, 1, 1), (64, 8, 4, 6), (100, 1, 1, 3), (256, 8, 4, 8), (256, 1, 1, 1), (512, 1, 1, 8), (512, 16, 4, 20),
         (1024, 1, 1, 8), (600, 6, 2, 17)]


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _far_below(T, E, dtype, offset, score):
    """Logits about `offset`; for a softmax two experts at 0, which a bias of -inf rules out; biases that tell the others
    apart."""
    l = _draw((T, E), dtype, 1, 0.5, offset)
    bias = torch.randperm(E, generator=_gen(2), device="cuda").float() * 0.125
    if score == "softmax":
        out = torch.tensor([1, E - 2], device="cuda")
        l[:, out] = 0.0
        bias[out] = -float("inf")
    return l, bias


def _distances(logits, ids, inside, top):
    """How far the chosen logits of a row lie below the largest of them, and how far the error bound reaches: a difference's
    rounding is u for each unit of it, exp 4 u, a few operations follow."""
    sel = np.where(inside, np.take_along_axis(logits, ids, 1), -np.inf)
    L = np.minimum(sel.max(1, keepdims=True), top)
    return np.where(inside, L - np.minimum(np.where(inside, sel, 0), top), 0)


@pytest.mark.parametrize("E,groups,kept,k", FORMS)
@pytest.mark.parametrize("score,dtype", [("softmax", "f32"), ("softmax", "bf16"), ("sigmoid", "f32"), ("sigmoid", "bf16")])
def test_weights_of_scores_below_the_normal_range(E, groups, kept, k, score, dtype):
    for T in (5, 700):
        for offset in (-80.0, -87.25, -88.0, -95.0, -150.0, -400.0):
            l, bias = _far_below(T, E, dtype, offset, score)
            for b in (bias, None) if score == "sigmoid" else (bias,):
                kw = dict(score=score, groups=groups, topk_groups=kept, scale=2.5)
                ids, w, counts = g.moe_route(l, k, bias=b, **kw)
                check_status()
                rids, rw, rc = ot.moe_route(_np(l), k, None if b is None else _np(b), **kw)
                assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(ids.cpu().numpy(), rids)
                d = np.abs(_distances(_np(l), rids, np.ones_like(rids, bool), 0.0 if score == "sigmoid" else np.inf))
                _within(w, rw, (40 + 2 * d + 2 * d.max(1, keepdims=True)) * U * rw, "f32", f"weights at {offset}")


@pytest.mark.parametrize("E,k", [(16, 1), (64, 6), (128, 3), (256, 8), (512, 32), (600, 8), (2048, 17)])
@pytest.mark.parametrize("score,dtype", [("softmax", "f32"), ("softmax", "bf16"), ("sigmoid", "f32"), ("sigmoid", "bf16")])
def test_gradient_of_scores_below_the_normal_range(E, k, score, dtype):
    T = 70
    for offset in (-80.0, -87.25, -88.0, -95.0, -150.0, -300.0):
        l, _ = _far_below(T, E, dtype, offset, score)
        ids = torch.argsort(torch.rand((T, E - 2), generator=_gen(3), device="cuda"), 1)[:, : min(k, E - 2)]
        ids = torch.where(ids == 1, E - 1, ids).to(torch.int32).contiguous()  # (of the experts that are far below)
        if score == "sigmoid":
            l[5, int(ids[5, 0])] = 3.0  # one that is not
        if k > 2:
            ids[1, 1] = ids[1, 0]
            ids[2, 0] = -1
        dw = _draw(ids.shape, "f32", 4, 100.0)
        mask = torch.arange(T, device="cuda") % 9 != 4
        kw = dict(score=score, renormalize=True, scale=2.5)
        got = g.moe_route_backward(l, ids, dw, token_mask=mask, **kw)
        check_status()
        n, at = _np(l), ids.cpu().numpy()
        want = ot.moe_route_backward(n, at, _np(dw), token_mask=_np(mask), **kw)
        # with p the weights over their sum: dlogits = p (dw - sum p dw), times 1 - s for a sigmoid
        inside = (at >= 0) & (at < E)
        at = np.where(inside, at, 0)
        d = np.abs(_distances(n, at, inside, 0.0 if score == "sigmoid" else np.inf))
        s = ot.route_scores(n, score)
        p = np.where(inside, np.take_along_axis(s, at, 1), 0.0)
        total = p.sum(1, keepdims=True)
        p = p / total
        a = np.abs(_np(dw)) * 2.5 * inside
        size = np.zeros((T, E))
        np.add.at(size, (np.arange(T)[:, None], at), p * (a + (p * a).sum(1, keepdims=True)) * 2)
        if score == "softmax":
            size = size + s * (p * a).sum(1, keepdims=True)
        # A score below 2^-126 is 0, or below that part of the largest where their sum is below 2^-60 (the largest is half of
        # what they are taken relative to, at least); it takes that much of its dw - sum p dw with it.
        gone = np.where(total >= 2.0 ** -60, 2.0 ** -126 / total, 2.0 ** -125)
        lost = np.zeros((T, E))
        np.add.at(lost, (np.arange(T)[:, None], at), gone * inside * (a + (p * a).sum(1, keepdims=True)))
        _within(got, want, (200 + 4 * d.max(1, keepdims=True)) * U * size + lost, dtype, f"dlogits at {offset}")
        assert not got[~mask].any()


@pytest.mark.parametrize("E,groups,kept,k", [(64, 1, 1, 6), (64, 8, 4, 6), (256, 8, 4, 8), (512, 1, 1, 8), (700, 1, 1, 8),
                                             (1024, 8, 2, 4)])
@pytest.mark.parametrize("score,dtype", [("softmax", "f32"), ("sigmoid", "f32"), ("sigmoid", "bf16")])
@pytest.mark.parametrize("level", [1e6, 1e9, 1e10, 1e12, -1e12, 1e16, 3e37])
def test_choice_with_biases_far_above_the_scores(E, groups, kept, k, score, dtype, level):
    """The choice is that of the sums in 64 bits, in every row alike: what they round off tells no experts apart."""
    for T in (40, 900):
        l = _draw((T, E), dtype, 1)
        kw = dict(score=score, groups=groups, topk_groups=kept)
        steps = torch.randint(0, 3, (E,), generator=_gen(2), device="cuda")
        for bias in (torch.full((E,), level, device="cuda"), level * (1 + steps * 2.0 ** -22)):
            ids, _, counts = g.moe_route(l, k, bias=bias, **kw)
            check_status()
            rids, _, rc = ot.moe_route(_np(l), k, _np(bias), **kw)
            assert np.array_equal(ids.cpu().numpy(), rids) and np.array_equal(counts.cpu().numpy(), rc)
