"""The gradient of a plain residual, h = x + scale gate f: df does not depend on f, whatever f holds."""

import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import DT, _draw, _strided

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


@pytest.mark.parametrize("N", [56, 128, 300, 512, 4096, 4099, 7168, 12288, 17000])
@pytest.mark.parametrize("sd,bd", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_df_is_free_of_f(N, sd, bd):
    M = 45
    for off in (0, 1):  # on one grid, and on none
        mat = lambda k, s, o=0: _strided((M, N), k, 0 if N % 8 else 8, o, seed=s)[0]  # noqa: E731
        f, dh = mat(bd, 1, off), mat(sd, 2)
        f[3, 5], f[4, N - 1], f[M - 1, 0] = float("inf"), float("nan"), -float("inf")
        gate = _draw((N,), "f32", 3, 0.3, 1.0)
        for a in (gate, None):
            dx, df = torch.empty((M, N), dtype=DT[sd], device="cuda"), torch.empty((M, N), dtype=DT[bd], device="cuda")
            dg = None if a is None else torch.empty(N, device="cuda")
            g.fp8g_residual_rms_norm_backward(None, dh, None, f, None, None, None, dx, df, dgate=dg, gate=a, scale=0.5)
            check_status()
            assert torch.equal(dx, dh)
            want = (dh.float() * (0.5 if a is None else 0.5 * a)).to(DT[bd])  # (0.5 is exact: one rounding, as the kernel's)
            assert torch.equal(df, want)
            if dg is not None:
                clean = [i for i in range(N) if i not in (0, 5, N - 1)]
                assert torch.isfinite(dg[clean]).all() and not torch.isfinite(dg[[0, 5, N - 1]]).any()
            # and with the norm of h in the way: the same bits with and without f
            x, h, dy, w = mat(sd, 4), mat(sd, 5), mat(bd, 6), _draw((N,), "f32", 7, 0.2, 1.0)
            r = (h.float().square().mean(1) + 1e-6).rsqrt()
            dw = [torch.empty(N, device="cuda") for _ in range(2)]
            out = [torch.empty_like(dx) for _ in range(2)], [torch.empty_like(df) for _ in range(2)]
            for i, ff in enumerate((f, None)):
                g.fp8g_residual_rms_norm_backward(dy, dh, h, ff, r, None, w, out[0][i], out[1][i], dw[i], gate=a, scale=0.5)
            assert torch.isfinite(out[1][0]).all()
            assert all(torch.equal(*p) for p in (out[0], out[1], dw))
