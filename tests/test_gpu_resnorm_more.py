"""The norms around a block at the borders of their forms: widths at which another number of lanes, CTAs or a cluster takes
a row, many rows a CTA, rows off the 16-byte grid by every distance, matrices that share no grid."""

import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import DT, _draw, _strided
from tests.test_gpu_train_ops import _check_norm, _check_norm_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _run(x, f, dy, dh, w, pw, gate, h, y, dx, df, sd, bd):
    M, N = x.shape
    rstd, rstd_f = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    g.fp8g_residual_rms_norm(x, f, w, h, y, rstd, rstd_f, gate, 0.5, True, pw)
    _check_norm(x, f, w, gate, 0.5, True, pw, (h, y, rstd, rstd_f), bd)
    dw, dg, dp = (torch.empty(N, device="cuda") for _ in range(3))
    g.fp8g_residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, w, dx, df, dw, dg, dp, gate, 0.5, True, pw)
    _check_norm_grad(dy, dh, h, f, rstd, rstd_f, w, gate, 0.5, True, pw, (dx, df, dw, dg, dp), sd, bd)
    check_status()


@pytest.mark.parametrize("N", [56, 57, 64, 65, 121, 128, 250, 256, 505, 512, 513, 4088, 4089, 4096, 4097, 8184, 8185, 8192, 8200,
                               16376, 16377, 16384])
@pytest.mark.parametrize("sd,bd", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_borders_of_the_forms(N, sd, bd):
    M = 1300 if N <= 520 else 170  # more rows than a wave of CTAs takes at once, for the narrow ones
    t = lambda k, s: _draw((M, N), k, s, 1.0)  # noqa: E731
    w, pw, gate = (_draw((N,), "f32", s, 0.2, 1.0) for s in (5, 6, 7))
    x, f = t(sd, 1), t(bd, 2)
    _run(x, f, t(bd, 3), t(sd, 4), w, pw, gate, torch.empty_like(x), torch.empty_like(f), torch.empty_like(x),
         torch.empty_like(f), sd, bd)


@pytest.mark.parametrize("pad", [1, 2, 3, 4, 5, 6, 7, 9])
@pytest.mark.parametrize("N", [40, 500, 1032, 12289])
def test_rows_off_the_grid_alike(pad, N):
    """All matrices' rows lie the same distance off the grid in every row; nothing beside them is written, and what lies
    there (NaN) is not taken in."""
    M = 700 if N < 600 else 330
    for sd, bd in (("f32", "bf16"), ("bf16", "bf16")):
        some = lambda k, s: _strided((M, N), k, pad, 0, seed=s)[0]  # noqa: E731
        outs = [_strided((M, N), k, pad, 0) for k in (sd, bd, sd, bd)]
        w, pw, gate = (_draw((N,), "bf16", s, 0.2, 1.0) for s in (5, 6, 7))
        (h, _), (y, _), (dx, _), (df, _) = outs
        _run(some(sd, 1), some(bd, 2), some(bd, 3), some(sd, 4), w, pw, gate, h, y, dx, df, sd, bd)
        for _, b in outs:
            assert torch.isnan(b[: M * (N + pad)].view(M, N + pad)[:, N:]).all() and torch.isnan(b[M * (N + pad):]).all()


@pytest.mark.parametrize("N", [24, 400, 1500, 9000, 17000])
def test_rows_that_share_no_grid(N):
    M = 300
    for sd, bd in (("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")):
        x, f = _strided((M, N), sd, 1, 1, seed=1)[0], _strided((M, N), bd, 2, 3, seed=2)[0]
        dy, dh = _strided((M, N), bd, 4, 0, seed=3)[0], _strided((M, N), sd, 5, 2, seed=4)[0]
        h, y, dx, df = (_strided((M, N), k, p, 1)[0] for k, p in ((sd, 0), (bd, 3), (sd, 8), (bd, 6)))
        w, pw, gate = (_draw((N,), "f32", s, 0.2, 1.0) for s in (5, 6, 7))
        _run(x, f, dy, dh, w, pw, gate, h, y, dx, df, sd, bd)


@pytest.mark.parametrize("N", [96, 4099, 7168, 12288])
def test_in_place(N):
    """h in x's place and dx in dh's give the bits of results apart."""
    M = 400
    x, f, dy, dh = _draw((M, N), "f32", 1), _draw((M, N), "bf16", 2), _draw((M, N), "bf16", 3), _draw((M, N), "f32", 4)
    w = _draw((N,), "f32", 5, 0.2, 1.0)
    h, y, rstd, rstd_f = g.residual_rms_norm(x, f, w, post_norm=True)
    dx, df, *_ = g.residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, w, post_norm=True)
    x2, y2, d2, df2 = x.clone(), torch.empty_like(y), dh.clone(), torch.empty_like(df)
    g.fp8g_residual_rms_norm(x2, f, w, x2, y2, post_norm=True)
    assert torch.equal(x2, h) and torch.equal(y2, y)
    g.fp8g_residual_rms_norm_backward(dy, d2, h, f, rstd, rstd_f, w, d2, df2, post_norm=True)
    assert torch.equal(d2, dx) and torch.equal(df2, df)
