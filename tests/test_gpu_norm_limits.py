"""Layer norm at the lengths next to its forms' limits, on the 16-byte grid and off it, contiguous and strided, where
what lies beside a row (padding, the rows before and after it, what earlier kernels left in shared memory) is not finite.

The bounds are those of test_gpu_block_ops.py: k = (N / 256 + 16) u covers a sum's additions, and the variance's
relative error is 2 k times the mean square of |x| + |mean| over the variance.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import block_ops as ob
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import DT, U, _check_norm_grads, _draw, _norm_bounds, _np, _strided, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _fill_shared(value):
    """An ordinary layer norm whose rows, all of `value`, take every SM's shared memory."""
    g.layer_norm(torch.full((2432, 7168), value, device="cuda"))


def _check_forward(y, mean, rstd, x, w, rows, yd):
    """The rows `rows` of a call's results."""
    N = x.shape[1]
    xn, wn = _np(x)[rows], _np(w)
    ry, rmean, rrstd = ob.layer_norm(xn, wn)
    k = (N / 256 + 16) * U
    ax = np.abs(xn)
    _within(mean[rows], rmean, k * ax.mean(1), "f32", "mean")
    var_err = 2 * k * ((ax + np.abs(rmean)[:, None]) ** 2).mean(1) * rrstd ** 2
    _within(rstd[rows], rrstd, (k + var_err) * rrstd, "f32", "rstd")
    _within(y[rows], ry, _norm_bounds(xn, wn, None, rmean, rrstd, N) + np.abs(ry) * var_err[:, None], yd, "y")


# the warp form ends at 57, 121 and 249 columns off the grid, a CTA's ring at 8185, a cluster's at 16377
LENGTHS = [*range(1, 10), 57, 58, 121, 122, *range(249, 267), 8185, 8186, 8193, 16377, 16378, 16383]


@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_rows_beside_anything(N, xd, yd):
    w = _draw((N,), "f32", 2, 0.3, 1.0)
    for M, pad in ((1, 0), (9, 0), (9, 1), (9, 3), (2, 8)):
        for bad in (float("nan"), float("inf"), 1e30):
            x, _ = _strided((M, N), xd, pad, 0, 5, std=2.0, mean=0.5)
            dy, _ = _strided((M, N), yd, pad, 0, 7, std=0.1)
            if M > 2:  # every second row starts and ends badly
                for t in (x, dy):
                    t[1::2, :8] = bad
                    t[1::2, -3:] = bad
            y, ybuf = _strided((M, N), yd, pad, 0)
            dx, dxbuf = _strided((M, N), xd, pad, 0)
            mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
            _fill_shared(bad)
            g.fp8g_layer_norm(x, w, None, y, mean, rstd)
            rows = np.arange(0, M, 2) if M > 2 else np.arange(M)
            _check_forward(y, mean, rstd, x, w, rows, yd)
            again = torch.empty_like(mean)
            _fill_shared(-1.0)
            g.fp8g_layer_norm(x, w, None, y, again, None)
            assert torch.equal(again[rows], mean[rows])  # the same bits, whatever lay in shared memory
            if pad:
                assert bool(torch.isnan(ybuf.view(-1)[N: N + pad]).all())
            _fill_shared(bad)
            g.fp8g_layer_norm_backward(dy, x, w, mean, rstd, dx, *torch.empty((2, N), device="cuda"))
            xn, dyn, mu, r = _np(x)[rows], _np(dy)[rows], _np(mean)[rows], _np(rstd)[rows]
            want = ob.layer_norm_backward(dyn, xn, _np(w), mu, r)[0]
            gw, hb = np.abs(dyn * _np(w)), (np.abs(xn) + np.abs(mu)[:, None]) * r[:, None]
            k = (N / 256 + 20) * U
            bound = 2 * k * r[:, None] * (gw + gw.mean(1, keepdims=True) + hb * (gw * hb).mean(1, keepdims=True))
            _within(dx[rows], want, bound, xd, "dx")
    check_status()


@pytest.mark.parametrize("N", [*range(249, 267), 8185, 8186, 16377])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_gradients_of_rows_beside_padding(N, xd):
    for M, pad in ((1, 0), (9, 0), (9, 3), (700, 1)):
        x, _ = _strided((M, N), xd, pad, 0, 5, std=2.0, mean=0.5)
        dy, _ = _strided((M, N), xd, pad, 0, 7, std=0.1)
        w = _draw((N,), "f32", 2, 0.3, 1.0)
        _, mean, rstd = g.layer_norm(x, w)
        dx, _ = _strided((M, N), xd, pad, 0)
        dw, db = torch.empty((2, N), device="cuda")
        _fill_shared(float("nan"))
        g.fp8g_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db)
        _check_norm_grads(dx, dw, db, dy, x, w, mean, rstd, xd)
    check_status()


@pytest.mark.parametrize("M,N", [(3000, 250), (3001, 252), (3000, 255), (3000, 263)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_many_rows_and_in_place(M, N, xd):
    x = _draw((M, N), xd, 3, 2.0, 0.5)
    w = _draw((N,), "f32", 2, 0.3, 1.0)
    x[5::7, 0] = float("nan")
    rows = np.setdiff1d(np.arange(M), np.arange(5, M, 7))
    _fill_shared(float("nan"))
    y, mean, rstd = g.layer_norm(x, w)
    _check_forward(y, mean, rstd, x, w, rows, xd)
    z = x.clone()
    g.fp8g_layer_norm(z, w, None, z)
    assert torch.equal(z[rows], y[rows])
    check_status()


# The ring takes differences from K, the mean of a row's first n = 240 to 256 values, so (K - mean)^2 <= N / n
# variances: the sums of squares are (1 + N / n) times the variance's own, and their roundings (k each, three of them:
# the squares' sum and twice the first sum's) weigh as much more.
@pytest.mark.parametrize("N", [264, 1000, 1003, 4096, 4099, 8192, 12288, 16384])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("far", [50.0, -3000.0])
def test_rows_that_start_far_from_their_mean(N, xd, far):
    x = _draw((5, N), xd, 11)
    x[:, :256] += far
    y, mean, rstd = g.layer_norm(x)
    xn = _np(x)
    ry, rmean, rrstd = ob.layer_norm(xn)
    k = (N / 256 + 16) * U
    var_err = 3 * k * (1 + N / 240)
    _within(mean, rmean, k * np.abs(xn).mean(1) + 2 * k / rrstd * (1 + N / 240) ** 0.5, "f32", "mean")
    _within(rstd, rrstd, (k + var_err) * rrstd, "f32", "rstd")
    bound = _norm_bounds(xn, None, None, rmean, rrstd, N) + 2 * k * (1 + N / 240) ** 0.5
    _within(y, ry, bound + np.abs(ry) * var_err, xd, "y")


# on the 16-byte grid a row's bits do not depend on how many rows the call has (off it they may: a single row starts on
# the grid whatever its stride)
@pytest.mark.parametrize("N", [8, 64, 512, 520, 1024, 1032, 4096, 8192, 8200, 16384, 20000])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("f32", "bf16")])
def test_a_row_on_the_grid_alone_has_the_same_bits(N, pad, xd, yd):
    x, _ = _strided((400, N), xd, pad, 0, 5, std=2.0, mean=0.5)
    dy, _ = _strided((400, N), yd, pad, 0, 7, std=0.1)
    w = _draw((N,), "f32", 2, 0.3, 1.0)
    y, mean, rstd = g.layer_norm(x, w, out_dtype=DT[yd])
    dx = g.layer_norm_backward(dy, x, w, mean, rstd)[0]
    for M in (1, 2, 9):
        some = g.layer_norm(x[:M], w, out_dtype=DT[yd])
        assert all(torch.equal(a, b[:M]) for a, b in zip(some, (y, mean, rstd)))
        assert torch.equal(g.layer_norm_backward(dy[:M], x[:M], w, mean[:M], rstd[:M])[0], dx[:M])
