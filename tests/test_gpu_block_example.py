"""The MoE block example: its loss falls, and one step's gradients agree with torch's automatic differentiation of the
same block in fp32, up to the FP8 rounding of its grouped GEMMs.

Rounding: e4m3 values are off by 2^-4 of themselves at most, about 2.6% in the root mean square; e5m2 ones by 2^-3,
about 5%.  A product's relative error in the 2-norm is the root of its factors' squares: 4% forward and 6% for the
gradients that pass through a grouped GEMM; twice that is allowed, and 1% for those that do not.
"""

import importlib.util
import os

import pytest
import torch

from tests.gpu_util import check_status, need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block_training.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_block_training", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _off(got, want):
    return float((got.float() - want).norm() / want.norm())


def test_the_loss_falls():
    need_gpu()
    log = _example().train(steps=8, tokens=600, hidden=512, experts=8, topk=2)
    assert all(l == l for row in log for l in row)
    assert log[-1][0] < 0.9 * log[0][0]
    check_status()


@pytest.mark.parametrize("T,hidden,E,topk,masked", [(300, 256, 4, 2, False), (513, 384, 8, 3, True)])
def test_gradients_agree_with_autograd(T, hidden, E, topk, masked):
    need_gpu()
    m = _example()
    block = m.MoEBlock(hidden, E, topk, seed=3, loss_coef=0.5)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, hidden), generator=gen, device="cuda")
    dout = torch.randn((T, hidden), generator=gen, device="cuda") / T
    mask = (torch.arange(T, device="cuda") % 10 < 8) if masked else None
    out, balance, saved = block.forward(x, mask)
    dx = block.backward(dout, saved)
    check_status()

    leaves = [t.clone().requires_grad_() for t in (x, block.weight, block.bias, block.router, block.experts)]
    x_, w_, b_, r_, e_ = leaves
    y = torch.nn.functional.layer_norm(x_, (hidden,), w_, b_, 1e-5)
    p = torch.softmax(y @ r_.t(), 1)
    ids, real = saved[5].long(), torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask
    wts = p.gather(1, ids)
    wts = wts / wts.sum(1, keepdim=True) * real[:, None]
    every = torch.einsum("eno,to->ten", e_, y)[torch.arange(T, device="cuda")[:, None], ids]
    ref = x_ + (every * wts[..., None]).sum(1)
    counts, tv = saved[7].float(), real.sum()
    ref_balance = 0.5 * E * (counts / (topk * tv) * p[real].sum(0) / tv).sum()
    ((ref * dout).sum() + ref_balance).backward()

    assert _off(out - x, (ref - x_).detach()) < 0.08
    assert _off(balance, ref_balance.detach().reshape(1)) < 0.01
    assert _off(dx, x_.grad) < 0.12
    assert _off(block.d_weight, w_.grad) < 0.12 and _off(block.d_bias, b_.grad) < 0.12
    assert _off(block.d_router, r_.grad) < 0.12
    assert _off(block.d_experts, e_.grad) < 0.12
