"""The oracle of the whole-block training operators, pinned: closed forms on tiny inputs, every gradient against central
differences of its own forward pass in 64 bits, and what the 8-bit AdamW states promise."""

import numpy as np
import pytest
import torch

from oracle import train_ops as ot
from tests.test_oracle_block_ops import _differences


def test_route_closed_form():
    # two groups of two: sums 0.5 + 0.5 and 0.9 + 0.01; the second expert of the best group is taken before the best of all
    s = np.array([[0.5, 0.5, 0.9, 0.01]])
    l = np.log(s / (1 - s))
    ids, w, counts = ot.moe_route(l, 2, groups=2, topk_groups=1)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5) and counts.tolist() == [1, 1, 0, 0]
    ids, w, _ = ot.moe_route(l, 2, bias=[0.0, 0.0, 0.0, 0.2], groups=2, topk_groups=1, renormalize=False, scale=2.0)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, [[1.8, 0.02]])  # the bias chooses, the score weighs
    ids, _, counts = ot.moe_route(l, 1, token_mask=[False])
    assert ids.tolist() == [[2]] and counts.sum() == 0


def test_route_ruled_out_experts():
    inf = np.inf
    l = np.array([[-inf, -inf, -inf, 1.0], [-inf] * 4, [0.0, np.nan, 1.0, 2.0]])
    ids, w, _ = ot.moe_route(l, 2, groups=2, topk_groups=1)
    assert ids[0].tolist() == [3, 2] and w[0].tolist() == [1.0, 0.0]  # its group has one expert, the other none
    assert ids[1].tolist() == [0, 1] and w[1].tolist() == [0.0, 0.0]
    assert ids[2].tolist() == [1, 0]
    ids, w, _ = ot.moe_route([[0.0, 0.0]], 2, bias=[-inf, 0.0])
    assert ids.tolist() == [[1, 0]] and w.tolist() == [[1.0, 0.0]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    l, c = rng.normal(size=(3, 6)), rng.normal(size=(3, 2))
    ids = np.array([[4, 0], [2, 2], [5, -1]])  # twice the same, and one outside
    mask = np.array([True, True, False])

    def f():
        s = ot.route_scores(l, score)
        sel = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
        w = sel / sel.sum(1, keepdims=True) if renorm else sel
        return float((1.7 * w * c * mask[:, None] * (ids >= 0)).sum())

    got = ot.moe_route_backward(l, ids, c, score, renorm, 1.7, mask)
    assert np.allclose(got, _differences(f, l), atol=1e-8)


def test_residual_norm_closed_form():
    h, y, rstd, rstd_f = ot.residual_rms_norm([[3.0, 4.0]], [[1.0, 7.0]], weight=[2.0, 1.0], scale=0.5, post_norm=True,
                                              post_weight=[5.0, 5.0], gate=[1.0, 0.0], eps=0.0)
    assert rstd_f[0] == 1 / 5.0 and np.allclose(h, [[3.5, 4.0]])
    assert np.allclose(y, np.array([[7.0, 4.0]]) * rstd[0]) and np.isclose(rstd[0], 1 / np.sqrt((3.5 ** 2 + 16) / 2))


@pytest.mark.parametrize("post,gated,parts", [(True, True, 3), (False, True, 3), (True, False, 3), (False, False, 3),
                                              (True, True, 1), (True, True, 2), (False, False, 0)])
def test_residual_norm_gradients_against_differences(post, gated, parts):
    rng = np.random.default_rng(2)
    x, f, cy, ch = (rng.normal(size=(3, 5)) for _ in range(4))
    w, p, a = (rng.normal(size=5) for _ in range(3))
    f = None if parts == 0 else f
    kw = dict(weight=w, gate=a if gated else None, scale=0.7, post_norm=post, post_weight=p if post else None)

    def value():
        h, y, _, _ = ot.residual_rms_norm(x, f, eps=1e-3, **kw)
        return float((h * ch).sum() * (parts != 1) + (y * cy).sum() * (parts != 2))

    h, _, rstd, rstd_f = ot.residual_rms_norm(x, f, eps=1e-3, **kw)
    dx, df, dw, dgate, dpost = ot.residual_rms_norm_backward(None if parts == 2 else cy, None if parts == 1 else ch, h, f,
                                                             rstd, rstd_f, **kw)
    assert np.allclose(dx, _differences(value, x), atol=1e-8)
    if parts != 2:
        assert np.allclose(dw, _differences(value, w), atol=1e-8)
    if f is not None:
        assert np.allclose(df, _differences(value, f), atol=1e-8)
        if gated:
            assert np.allclose(dgate, _differences(value, a), atol=1e-8)
        if post:
            assert np.allclose(dpost, _differences(value, p), atol=1e-8)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(3)
    gu, c = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4))
    assert np.isclose(ot.swiglu([[1.0, 3.0]])[0, 0], 3.0 / (1 + np.exp(-1.0)))
    got = ot.swiglu_backward(c, gu)
    assert np.allclose(got, _differences(lambda: float((ot.swiglu(gu) * c).sum()), gu), atol=1e-8)


def test_adamw_agrees_with_torchs():
    gen = torch.Generator().manual_seed(0)
    p = torch.randn(40, generator=gen, dtype=torch.float64).requires_grad_()
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.9), eps=1e-6, weight_decay=0.3)
    q, m, v = p.detach().numpy().copy(), np.zeros(40), np.zeros(40)
    for t in range(1, 6):
        g = torch.randn(40, generator=gen, dtype=torch.float64)
        p.grad = g
        opt.step()
        q, m, v = ot.adamw(q, g.numpy(), m, v, t, 0.01, 0.8, 0.9, 1e-6, 0.3)
    assert np.allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-12)


def test_states_lie_between_neighbouring_codes():
    rng = np.random.default_rng(4)
    x = (rng.normal(size=1000) * 10.0 ** rng.uniform(-6, 0, size=1000)).astype(np.float32)
    codes, scales = ot.encode_states(x, 7, False)
    got = ot.state_values(codes, scales).astype(np.float64)
    s = np.repeat(scales, 128)[:1000].astype(np.float64)
    y = np.abs(x) / s
    unit = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    assert np.all(np.abs(got - x) <= unit * s * (1 + 1e-5))
    assert scales.shape == (8,) and np.all(np.abs(got).reshape(-1)[:896].reshape(7, 128).max(1) > 0)


def test_states_are_right_on_the_average_of_the_steps():
    """The mean of the codes' values over 512 steps: a value's place between two codes is met to 1/128 of their distance
    (the discrepancy of such a sequence falls as log(n) / n: about 6 / 512)."""
    x = np.linspace(0.01, 1.0, 128).astype(np.float32)
    values = np.array([ot.state_values(*ot.encode_states(x, t, False)) for t in range(512)]).astype(np.float64)
    y = x / (1.0 / 448.0)
    unit = 2.0 ** (np.floor(np.log2(y)) - 3) / 448.0
    assert np.max(np.abs(values.mean(0) - x) / unit) < 1 / 64


def test_eight_bit_states_follow_a_fall_of_the_gradients():
    """All gradients but a block's first fall to a quarter: after 3000 steps at beta2 = 0.999 (0.05 of the old square is
    left: v = 0.05 + 0.95 / 16 of it) the roots have followed on the average.  Rounded to the nearest they could not: a
    step changes them by less than 0.05%, half a code's distance is 3%."""
    g = np.ones(128, np.float32)
    root = np.ones(128, np.float32)
    g[1:] = 0.25
    codes, scales = ot.encode_states(root, 0, True)
    m = np.zeros(128, np.float32)
    for t in range(1, 3001):
        m, root = ot.adamw_states(g, m, ot.state_values(codes, scales), 0.9, 0.999)
        codes, scales = ot.encode_states(root, t, True)
    want = np.sqrt(0.999 ** 3000 + (1 - 0.999 ** 3000) / 16)
    assert abs(ot.state_values(codes, scales)[1:].mean() / want - 1) < 0.1


def test_roots_that_are_not_zero_keep_a_code():
    x = np.array([1.0, 1e-9, 0.0, 1e-30], np.float32)
    codes, _ = ot.encode_states(x, 3, True)
    assert codes.tolist()[1:] == [1, 0, 1]
    codes, scales = ot.encode_states(np.full(3, 1e-20, np.float32), 3, True)
    assert codes.tolist() == [0, 0, 0] and scales.tolist() == [0.0]
