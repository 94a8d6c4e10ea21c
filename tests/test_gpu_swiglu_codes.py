"""The gated activation's codes and scales against the unfused quantiser's rule applied to the fp32 products: s = fp32(amax / 448),
codes of the rounded quotients fp32(h / s).  Gates of 33 and more have s(g) = 1 in fp32, so h = g u is exact there (two
significands of 8 bits)."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle.quantize import quantize_1x128
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import U, _draw

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _masked(gu):
    """The masked form's codes and scales of the same rows, three experts of a third each."""
    M, F = gu.shape[0] // 3 * 3, gu.shape[1] // 2
    q = torch.zeros((3, M // 3, F), dtype=torch.uint8, device="cuda")
    s = torch.zeros((F // 128, (M + 3) // 4 * 4), device="cuda")
    g.fp8_swiglu_quantize_1x128_masked(gu[:M].contiguous().view(3, M // 3, 2 * F), q, s,
                                       torch.full((3,), M // 3, dtype=torch.int32, device="cuda"))
    return q.view(M, F), s[:, :M]


def _compare(gate, up):
    gu = torch.cat([gate, up], 1).bfloat16()
    M, F = gate.shape
    assert torch.equal(gu.float(), torch.cat([gate, up], 1))
    want_q, want_s = quantize_1x128((gate * up).cpu().numpy())
    q, s, h = g.swiglu_quantize_1x128(gu, keep=True)
    check_status()
    assert np.array_equal(s[:, :M].cpu().numpy().T, want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert torch.equal(h, (gate * up).bfloat16())
    mq, ms = _masked(gu)
    n = len(mq)
    assert torch.equal(mq, q[:n]) and torch.equal(ms, s[:, :n])


def test_codes_where_the_quotient_lies_between_two_codes():
    """Rows of gate k with a largest up of 448 have the scale k, and ups halfway between two codes, whose quotients are
    exactly that: they go to the even code."""
    ups = [448.0] + [m * 2.0 ** e for e in range(-9, 5) for m in (17, 19, 21, 23, 25, 27, 29, 31)]
    ups = ups + [-u for u in ups]
    up = torch.tensor((ups + [0.0] * (256 - len(ups)))[:256], device="cuda").expand(223, 256).contiguous()
    up[:, 0] = up[:, 128] = 448.0
    _compare(torch.arange(33.0, 256.0, device="cuda")[:, None].expand(223, 256).contiguous(), up)


@pytest.mark.parametrize("std", [1e-20, 1e-3, 1.0, 1e30])
def test_codes_of_products_that_fp32_holds(std):
    gate = (_draw((600, 384), "f32", 1).abs() * 30 + 40).bfloat16().float()
    _compare(gate, _draw((600, 384), "bf16", 2, std).float())


def test_a_block_with_a_product_beyond_fp32():
    """Its scale is infinite, so finite values become 0 and the infinite one has no code but NaN; the blocks beside it do
    not feel it."""
    gate = torch.full((3, 256), 64.0, device="cuda")
    up = _draw((3, 256), "bf16", 1).float()
    gate[1, 7], up[1, 7] = 2.0 ** 100, -2.0 ** 100
    gu = torch.cat([gate, up], 1).bfloat16()
    q, s, h = g.swiglu_quantize_1x128(gu, keep=True)
    check_status()
    rest = [0, 2]
    want_q, want_s = quantize_1x128((gate * up)[rest].cpu().numpy())
    got = q.cpu().numpy()
    assert np.array_equal(got[rest], want_q) and np.array_equal(s[:, rest].cpu().numpy().T, want_s)
    want_q, want_s = quantize_1x128((gate * up)[1:2, 128:].cpu().numpy())
    assert np.array_equal(got[1:2, 128:], want_q) and float(s[1, 1]) == want_s[0, 0]
    assert float(s[0, 1]) == float("inf") and got[1, 7] & 0x7F == 0x7F
    assert not (np.delete(got[1, :128], 7) & 0x7F).any()
    assert float(h[1, 7]) == -float("inf") and int(torch.isinf(h).sum()) == 1
    mq, ms = _masked(gu)
    assert torch.equal(mq, q) and torch.equal(ms, s[:, :3])


def test_blocks_of_zeros_and_of_what_is_no_number():
    """A block of zeros, of either sign, has the codes 0x00; one of NaN alone keeps them."""
    gu = torch.full((4, 256), -0.0, dtype=torch.bfloat16, device="cuda")
    gu[1, :128] = -1.0  # h = -0
    gu[2, :128], gu[2, 128:] = 2.0, float("nan")
    gu[3, :128], gu[3, 200] = 2.0, float("nan")
    q, s, _ = g.swiglu_quantize_1x128(gu)
    check_status()
    assert not q[:2].any() and s[0, :4].tolist() == [0.0] * 4
    assert (q[2] & 0x7F == 0x7F).all() and int((q[3] & 0x7F == 0x7F).sum()) == 1 and int(q[3, 72]) & 0x7F == 0x7F


def test_the_gates_own_error_does_not_grow_with_them():
    """The scale of a block of equal products is their fp32 value over 448.  The exponential is off by 2 units in the last
    place (4 u) and the 1.5 u that the next term of e^(g c) has at g = -87; its product, 1 + exp, two products and the scale
    add a rounding each, the reciprocal a unit (2 u): 12.5 u.  (s(g) below 2^-126, of gates below -87.3, is 0.)"""
    gates = torch.cat([torch.linspace(-87.0, 99.0, 500), torch.linspace(-3.0, 3.0, 500)]).bfloat16().double()
    gu = torch.cat([gates[:, None].expand(-1, 128), torch.full((1000, 128), 64.0, dtype=torch.float64)], 1).bfloat16().cuda()
    _, s, _ = g.swiglu_quantize_1x128(gu)
    want = (gates / (1.0 + torch.exp(-gates)) * 64.0 / 448.0).abs().numpy()
    got = s[0, :1000].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 12.5 * U * 1.01 * want + 2.0 ** -149)
