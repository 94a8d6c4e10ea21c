"""Softmax rows that fp32 leaves in doubt, at numbers of experts whose warps do not divide a CTA's: some warps of the CTA's end
have no row (csrc/shares.cuh)."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import train_ops as ot
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import _gen, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [70, 3000])
@pytest.mark.parametrize("E", [65, 96, 160, 200, 224, 320, 448])
def test_rows_in_doubt(T, E):
    need_gpu()
    base = torch.randn((T, 1), generator=_gen(5), device="cuda")
    near = base * (1 + torch.randint(0, 5, (T, E), generator=_gen(6), device="cuda") * 2.0 ** -23)
    bias = torch.zeros(E, device="cuda")
    ids, w, counts = g.moe_route(near, 4, bias=bias, score="softmax")
    check_status()
    want, _, rc = ot.moe_route(_np(near), 4, _np(bias), score="softmax")
    assert np.array_equal(ids.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), rc)
    assert np.allclose(_np(w), 0.25, rtol=1e-5, atol=0)  # (the chosen logits of a row differ by 4 2^-23 |base| at most)
