"""The oracle of the training operators, pinned: closed forms on tiny inputs, and every gradient against central
differences of its own forward pass in 64 bits."""

import numpy as np
import pytest

from oracle import block_ops as ob


def _differences(f, x, step=1e-5):
    """The gradient of the scalar f at x by central differences (error: about step^2 and 1e-16 / step)."""
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + step
        hi = f()
        flat[i] = keep - step
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * step)
    return g


def test_layer_norm_closed_form():
    y, mean, rstd = ob.layer_norm([[1.0, 3.0], [5.0, 5.0]], weight=[2.0, 2.0], bias=[0.5, 0.0], eps=0.0 + 1e-300)
    assert mean.tolist() == [2.0, 5.0]
    assert y[0].tolist() == [-1.5, 2.0] and y[1].tolist() == [0.5, 0.0]
    assert rstd[0] == 1.0


@pytest.mark.parametrize("weighted", [True, False])
def test_layer_norm_gradient_against_differences(weighted):
    rng = np.random.default_rng(0)
    x, c = rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    w, b = rng.normal(size=5), rng.normal(size=5)

    def f():
        return float((ob.layer_norm(x, w if weighted else None, b)[0] * c).sum())

    _, mean, rstd = ob.layer_norm(x)
    dx, dw, db = ob.layer_norm_backward(c, x, w if weighted else None, mean, rstd)
    assert np.allclose(dx, _differences(f, x), atol=1e-8)
    if weighted:
        assert np.allclose(dw, _differences(f, w), atol=1e-8)
    assert np.allclose(db, _differences(f, b), atol=1e-8)


def test_gate_closed_forms():
    # uniform logits: ties go to the lowest index; every expert equally likely
    ids, w, counts, loss = ob.moe_gate(np.zeros((4, 8)), 2, renormalize=True, loss_coef=1.0)
    assert ids.tolist() == [[0, 1]] * 4 and np.all(w == 0.5)
    assert counts.tolist() == [4, 4, 0, 0, 0, 0, 0, 0]
    assert loss == pytest.approx(1.0)  # E sum_e f_e / E = 1
    # one expert takes everything: E f P = E
    l = np.full((3, 4), -np.inf)
    l[:, 2] = 1.0
    ids, w, counts, loss = ob.moe_gate(l, 1, loss_coef=1.0)
    assert ids.tolist() == [[2]] * 3 and np.all(w == 1.0) and loss == pytest.approx(4.0)
    # a masked row: zeros, and it is not counted
    ids, w, counts, loss = ob.moe_gate(np.zeros((2, 4)), 2, token_mask=[1, 0])
    assert w[1].tolist() == [0.0, 0.0] and counts.sum() == 2
    # nothing but -inf
    ids, w, counts, loss = ob.moe_gate(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]] and loss == 0.0


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("masked", [True, False])
def test_gate_gradient_against_differences(renorm, masked):
    rng = np.random.default_rng(1)
    l, c = rng.normal(size=(5, 6)), rng.normal(size=(5, 3))
    l[0, 4] = -np.inf
    mask = np.array([1, 0, 1, 1, 1]) if masked else None
    ids, _, counts, _ = ob.moe_gate(l, 3, renorm, 0.5, mask)

    def f():
        i, w, n, loss = ob.moe_gate(l, 3, renorm, 0.5, mask)
        assert np.array_equal(i, ids)
        return float((w * c).sum()) + 1.7 * loss

    got = ob.moe_gate_backward(l, ids, counts, c, 1.7, renorm, 0.5, mask)
    free = np.isfinite(l)
    want = np.zeros_like(l)
    for t, e in zip(*np.nonzero(free)):
        keep = l[t, e]
        l[t, e] = keep + 1e-5
        hi = f()
        l[t, e] = keep - 1e-5
        lo = f()
        l[t, e] = keep
        want[t, e] = (hi - lo) / 2e-5
    assert np.allclose(got, want, atol=1e-8)


def test_combine_and_its_gradient():
    rng = np.random.default_rng(2)
    D, w, c = rng.normal(size=(6, 4)), rng.normal(size=(3, 2)), rng.normal(size=(3, 4))
    rows = np.array([[0, 5], [2, -1], [-1, -1]])
    out = ob.moe_combine(D, rows, w, residual=np.ones((3, 4)))
    assert np.allclose(out[0], 1 + w[0, 0] * D[0] + w[0, 1] * D[5]) and np.all(out[2] == 1.0)

    def f():
        return float((ob.moe_combine(D, rows, w) * c).sum())

    dD, dw = ob.moe_combine_backward(c, D, rows, w)
    assert np.allclose(dD, _differences(f, D), atol=1e-8)
    assert np.allclose(dw, _differences(f, w), atol=1e-8)


def test_clip_closed_form():
    norm, out = ob.clip_grad_norm([[3.0], [4.0, 0.0]], 1.0, eps=0.0)
    assert norm == 5.0 and np.allclose(out[0], [0.6]) and np.allclose(out[1], [0.8, 0.0])
    norm, out = ob.clip_grad_norm([[3.0]], 10.0)
    assert out[0].tolist() == [3.0]
