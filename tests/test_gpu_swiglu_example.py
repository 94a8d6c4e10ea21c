"""The gated MoE block example: it runs, and one step's gradients agree with torch's automatic differentiation of the same
block in fp32, up to the FP8 rounding of its grouped GEMMs.

Rounding: e4m3 values are off by 2^-4 of themselves at most, about 2.6% in the root mean square; e5m2 ones by 2^-3, about
5%.  A product's relative error in the 2-norm is the root of its factors' squares.  Forward: two products of two e4m3
factors each, 4% and 4%, which the activation about doubles for the first (its gates and ups are both off): 9%.  A
gradient passes two products with an e5m2 factor, 6% each, and is formed from forward values that are off by 9%:
the root of the squares is 13%; twice that is allowed, and for the norms' and the router's too, which sum over tokens.
"""

import importlib.util
import os

import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from tests.gpu_util import check_status, need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_swiglu_training.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_swiglu_training", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _off(got, want):
    return float((got.float() - want).norm() / want.norm())


def test_it_runs():
    need_gpu()
    log = _example().train(steps=4, tokens=600, hidden=512, inner=256, experts=8, topk=2)
    assert len(log) == 4 and all(v == v and v < 1e4 for row in log for v in row)
    check_status()


@pytest.mark.parametrize("T,hidden,inner,E,topk,groups,masked", [(300, 256, 128, 8, 2, 4, False), (513, 384, 256, 16, 4, 4, True)])
def test_gradients_agree_with_autograd(T, hidden, inner, E, topk, groups, masked):
    need_gpu()
    m = _example()
    block = m.GatedMoEBlock(hidden, inner, E, topk, groups=groups, topk_groups=2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    block.bias.copy_(torch.randn(E, generator=gen, device="cuda") * 0.05)
    x = torch.randn((T, hidden), generator=gen, device="cuda")
    dz = (torch.randn((T, hidden), generator=gen, device="cuda") / T).bfloat16()
    mask = (torch.arange(T, device="cuda") % 10 < 8) if masked else None
    z, saved = block.forward(x, mask)
    dx = block.backward(dz, saved)
    check_status()

    x_ = x.clone().requires_grad_()
    leaves = [p.float().clone().requires_grad_() for p in block.params]
    w_in, w_out, router, w, post, gate, w_next = leaves
    rms = lambda t: t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    y = rms(x_) * w
    score = torch.sigmoid(y @ router.t())
    ids = saved[4].long()
    p = score.gather(1, ids)
    p = p / p.sum(1, keepdim=True)
    if mask is not None:
        p = p * mask[:, None]
    gu = torch.einsum("eno,to->ten", w_in, y)[torch.arange(T, device="cuda")[:, None], ids]
    a = torch.nn.functional.silu(gu[..., :inner]) * gu[..., inner:]
    each = torch.einsum("tkn,tkon->tko", a, w_out[ids])
    f = (each * p[..., None]).sum(1)
    h = x_ + block.scale * gate * (rms(f) * post)
    ref = rms(h) * w_next
    (ref * dz.float()).sum().backward()

    assert _off(z, ref.detach()) < 0.09
    assert _off(dx, x_.grad) < 0.26
    for got, leaf in zip(block.grads, leaves):
        assert _off(got, leaf.grad) < 0.26


def test_a_replayed_step_is_the_eager_one():
    """Forward, backward and update of the operators together, captured and replayed: the same bits."""
    need_gpu()
    m = _example()
    x = torch.randn((256, 256), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    dz = torch.full((256, 256), 1e-3, device="cuda", dtype=torch.bfloat16)

    def step(block):
        _, saved = block.forward(x)
        block.backward(dz, saved)
        return block.update(1e-3, 0.5, saved[6])

    a, b = (m.GatedMoEBlock(256, 128, 8, 2, seed=7) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a)  # (gives the stream its workspaces)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step(a)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for _ in range(3):
        want = step(b)
    assert int(a.opt.step) == int(b.opt.step) == 3
    assert torch.equal(norm, want) and torch.equal(a.bias, b.bias)
    for p, q in zip(a.opt.tensors, b.opt.tensors):
        assert torch.equal(p, q)
    check_status()
