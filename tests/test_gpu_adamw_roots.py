"""AdamW's 8-bit states of second moments: a block with one value has its root over 448 as the scale.  The root is the rounded
one or, for about one value in 2^20, the float next to it."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import train_ops as ot
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import _draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("std", [1e-12, 0.01, 1e10])
def test_roots_are_the_rounded_ones_or_next_to_them(std):
    need_gpu()
    blocks = 1 << 18
    d = torch.zeros((blocks, 128), device="cuda")
    d[:, 5] = _draw((blocks,), "f32", 1, std)
    p = torch.zeros_like(d)
    opt = g.AdamWList([p], [d], state_bits=8, weight_decay=0.0)
    g.adamw_step(opt, 1e-2)
    check_status()
    zero = np.zeros(blocks, np.float32)
    _, root = ot.adamw_states(d[:, 5].cpu().numpy(), zero, zero, 0.9, 0.999)
    want = np.where(root >= np.float32(2.0 ** -60), root * (np.float32(1) / np.float32(448)), np.float32(0))
    got = opt.v_scales[0].cpu().numpy()
    # a unit of the root (2^-23 of it at most) and the product's rounding on either side (2^-24 each)
    assert np.all(np.abs(got.astype(np.float64) - want) <= 2.0 ** -22 * want)
    assert np.mean(got != want) <= 1e-4
    codes = opt.v[0].view(blocks, 128).cpu().numpy()
    assert np.array_equal(codes[:, 5], np.where(want > 0, 0x7E, 0)) and not np.delete(codes, 5, 1).any()
