"""The gate's weights are as exact for experts far below the row's largest as for those near it.

Logits are multiples of 1/4 here, so their differences are exact.  With u = 2^-24: a selected expert's exponential is off
by 4 u (the instruction's own bound), the row's sum by the 4 u of its terms, by their exponents' rounding (1.3 u for each
unit below the largest, weighted by the term itself: under u) and by 13 additions one after another; the reciprocal by 2 u,
the product by u.  25 u in all; renormalised, the picks' sum stands for the row's."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import block_ops as ob
from tests.gpu_util import need_gpu
from tests.test_gpu_block_ops import DT, U, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,topk", [(60, 8, 8), (60, 32, 32), (300, 64, 16), (40, 256, 32), (5000, 256, 32),
                                      (30, 384, 32), (9, 1500, 32)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [False, True])
def test_weights_far_below_the_largest(T, E, topk, xd, renorm):
    need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(E)
    logits = (torch.randint(-160, -60, (T, E), generator=gen, device="cuda") / 4.0).to(DT[xd])
    spread = torch.randint(0, 160, (T, topk), generator=gen, device="cuda") / 4.0
    cols = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :topk]
    logits.scatter_(1, cols, (40.0 - spread).to(DT[xd]))  # the selected ones: up to 40 below the largest
    ids, w, _, _ = g.moe_gate(logits, topk, renormalize=renorm)
    rids, rw, _, _ = ob.moe_gate(_np(logits), topk, renorm)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert float((np.abs(_np(w) - rw) / rw).max()) <= 25 * U
