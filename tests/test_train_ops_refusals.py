"""The whole-block training operators' argument checks, in the library (before anything is launched) and in the binding;
and the calls that have nothing to do.  No GPU needed."""

import ctypes

import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from moe_grouped_gemm_block_gb300.train_ops import _Tensor
from tests.test_block_ops_refusals import BIG, P, _args

INVALID, ALIGN = 1, 2
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return g.lib()


ROUTE = dict(l=P, d=1, T=4, E=16, ldl=16, k=2, bias=P, score=0, groups=4, kept=2, renorm=1, scale=1.0, mask=None, ids=P,
             w=P, counts=P, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=2), INVALID), (dict(E=0), INVALID), (dict(E=2049, ldl=2049, groups=1, kept=1), INVALID), (dict(ldl=15), INVALID),
    (dict(k=0), INVALID), (dict(k=33, E=64, ldl=64), INVALID), (dict(k=9), INVALID), (dict(score=2), INVALID),
    (dict(groups=3), INVALID), (dict(groups=0), INVALID), (dict(groups=64, E=64, ldl=64), INVALID), (dict(kept=0), INVALID),
    (dict(kept=5), INVALID), (dict(renorm=2), INVALID), (dict(scale=NAN), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 30, k=4), INVALID), (dict(l=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID),
    (dict(counts=None), INVALID), (dict(T=0, counts=None), INVALID),
    (dict(l=P + 2), ALIGN), (dict(bias=P + 1), ALIGN), (dict(ids=P + 2), ALIGN), (dict(counts=P + 2), ALIGN),
])
def test_route(lib, kw, want):
    assert lib.fp8g_moe_route(*_args(ROUTE, kw)) == want


ROUTE_BWD = dict(l=P, d=1, T=4, E=16, ldl=16, k=2, score=0, renorm=1, scale=1.0, mask=None, ids=P, dw=P, dl=P, ldd=16,
                 s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=2), INVALID), (dict(ldd=15), INVALID), (dict(k=17), INVALID), (dict(score=-1), INVALID), (dict(ids=None), INVALID),
    (dict(dw=None), INVALID), (dict(dl=None), INVALID), (dict(scale=NAN), INVALID), (dict(dl=P + 2), ALIGN),
    (dict(dw=P + 2), ALIGN), (dict(T=0, l=None, ids=None, dw=None, dl=None), 0),
])
def test_route_backward(lib, kw, want):
    assert lib.fp8g_moe_route_backward(*_args(ROUTE_BWD, kw)) == want


NORM = dict(x=P, ldx=64, f=P, ldf=64, sd=1, bd=0, M=4, N=64, post=1, pw=P, gate=P, scale=1.0, w=P, wd=1, eps=1e-6, h=P,
            ldh=64, y=P, ldy=64, rf=P, r=P, s=None)
NO_BLOCK = dict(f=None, h=None, post=0, pw=None, gate=None)


@pytest.mark.parametrize("kw,want", [
    (dict(sd=2), INVALID), (dict(bd=-1), INVALID), (dict(wd=3), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(M=1 << 31), INVALID), (dict(ldx=63), INVALID), (dict(ldf=8), INVALID), (dict(ldh=8), INVALID), (dict(ldy=8), INVALID),
    (dict(post=2), INVALID), (dict(post=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(x=None), INVALID), (dict(h=None, y=None), INVALID), (dict(f=None), INVALID), ({**NO_BLOCK, "gate": P}, INVALID),
    ({**NO_BLOCK, "post": 1}, INVALID), ({**NO_BLOCK, "h": P}, INVALID),
    (dict(x=P + 2), ALIGN), (dict(f=P + 1), ALIGN), (dict(w=P + 2), ALIGN), (dict(r=P + 2), ALIGN), (dict(h=P + 2), ALIGN),
    (dict(M=0, x=None), 0), ({**NO_BLOCK, "M": 0}, 0),
])
def test_residual_norm(lib, kw, want):
    assert lib.fp8g_residual_rms_norm(*_args(NORM, kw)) == want


NORM_BWD = dict(dy=P, lddy=64, dh=P, lddh=64, h=P, ldh=64, f=P, ldf=64, sd=1, bd=0, M=4, N=64, post=1, pw=P, gate=P,
                scale=1.0, w=P, wd=1, rf=P, r=P, dx=P, lddx=64, df=P, lddf=64, dw=P, dg=P, dp=P, ws=P, wsb=BIG, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(sd=2), INVALID), (dict(lddy=8), INVALID), (dict(lddh=8), INVALID), (dict(ldh=8), INVALID), (dict(ldf=8), INVALID),
    (dict(lddx=8), INVALID), (dict(lddf=8), INVALID), (dict(dx=None), INVALID), (dict(dy=None, dh=None, dw=None), INVALID),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(r=None), INVALID), (dict(rf=None), INVALID),
    (dict(f=None), INVALID), (dict(post=0), INVALID), (dict(df=None), INVALID), (dict(gate=None), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=64), INVALID), (dict(f=None, post=0, pw=None, dp=None), INVALID),
    (dict(ws=P + 8), ALIGN), (dict(dw=P + 2), ALIGN), (dict(dx=P + 2), ALIGN), (dict(df=P + 1), ALIGN),
    (dict(M=0, dw=None, dg=None, dp=None, ws=None), 0),
])
def test_residual_norm_backward(lib, kw, want):
    assert lib.fp8g_residual_rms_norm_backward(*_args(NORM_BWD, kw)) == want


def test_residual_norm_workspace(lib):
    n = ctypes.c_int64()
    assert lib.fp8g_residual_rms_norm_backward_workspace(0, 64, ctypes.byref(n)) == 0 and n.value >= 16
    assert lib.fp8g_residual_rms_norm_backward_workspace(5000, 7168, ctypes.byref(n)) == 0 and n.value >= 2 * 7168 * 4
    assert lib.fp8g_residual_rms_norm_backward_workspace(-1, 64, ctypes.byref(n)) == INVALID
    assert lib.fp8g_residual_rms_norm_backward_workspace(4, 0, ctypes.byref(n)) == INVALID
    assert lib.fp8g_residual_rms_norm_backward_workspace(4, 4, None) == INVALID


GLU = dict(gu=P, M=4, F=128, ldgu=256, q=P, ldq=128, sA=P, ld_sa=4, h=P, ldh=128, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(F=0), INVALID), (dict(F=64, ldgu=256), INVALID), (dict(F=132, ldgu=264, q=None), INVALID),
    (dict(ldgu=248), INVALID), (dict(q=None, h=None), INVALID), (dict(sA=None), INVALID), (dict(ldq=112), INVALID),
    (dict(ld_sa=0), INVALID), (dict(ldh=120), INVALID), (dict(gu=None), INVALID), (dict(M=1 << 31, ld_sa=1 << 32), INVALID),
    (dict(gu=P + 8), ALIGN), (dict(q=P + 8), ALIGN), (dict(sA=P + 4), ALIGN), (dict(h=P + 2), ALIGN), (dict(ldgu=260), ALIGN),
    (dict(ldq=136), ALIGN), (dict(ld_sa=6), ALIGN), (dict(ldh=132), ALIGN), (dict(M=0, gu=None), 0),
])
def test_swiglu(lib, kw, want):
    assert lib.fp8_swiglu_quantize_1x128(*_args(GLU, kw)) == want


GLU_MASKED = dict(gu=P, E=2, cap=4, F=128, counts=P, q=P, sA=P, ld_sa=8, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(E=0), INVALID), (dict(E=65536, ld_sa=1 << 20), INVALID), (dict(cap=-1), INVALID), (dict(F=64), INVALID),
    (dict(ld_sa=4), INVALID), (dict(counts=None), INVALID), (dict(q=None), INVALID), (dict(gu=None), INVALID),
    (dict(sA=P + 8), ALIGN), (dict(counts=P + 2), ALIGN), (dict(ld_sa=10), ALIGN), (dict(cap=0, gu=None), 0),
])
def test_swiglu_masked(lib, kw, want):
    assert lib.fp8_swiglu_quantize_1x128_masked(*_args(GLU_MASKED, kw)) == want


GLU_BWD = dict(dh=P, lddh=128, gu=P, M=4, F=128, ldgu=256, dgu=P, lddgu=256, h=P, ldh=128, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(F=100, lddh=104), INVALID), (dict(lddh=120), INVALID), (dict(ldgu=128), INVALID),
    (dict(lddgu=128), INVALID), (dict(ldh=8), INVALID), (dict(dh=None), INVALID), (dict(dgu=None), INVALID),
    (dict(dh=P + 2), ALIGN), (dict(dgu=P + 8), ALIGN), (dict(lddh=130), ALIGN), (dict(M=0, dh=None, gu=None, dgu=None), 0),
])
def test_swiglu_backward(lib, kw, want):
    assert lib.fp8g_swiglu_backward(*_args(GLU_BWD, kw)) == want


TENSOR = dict(param=P, grad=P, m=P, v=P, m_scale=P, v_scale=P, master=None, numel=8, weight_decay=0.0, param_dtype=1,
              grad_dtype=0, reserved=0)
ADAM = dict(bits=8, lr=1e-3, lr_dev=None, b1=0.9, b2=0.99, eps=1e-8, step=P, norm=P, max_norm=1.0, norm_eps=0.0, ws=P, wsb=64,
            s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(bits=16), INVALID), (dict(lr=-1.0), INVALID), (dict(lr=NAN), INVALID), (dict(b1=1.0), INVALID), (dict(b2=-0.1), INVALID),
    (dict(b2=NAN), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(step=None), INVALID),
    (dict(max_norm=-1.0), INVALID), (dict(max_norm=NAN), INVALID), (dict(norm_eps=-1.0), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=32), INVALID), (dict(numel=-1), INVALID), (dict(numel=1 << 41), INVALID), (dict(param=None), INVALID),
    (dict(grad=None), INVALID), (dict(m=None), INVALID), (dict(v_scale=None), INVALID), (dict(param_dtype=2), INVALID),
    (dict(grad_dtype=-1), INVALID), (dict(master=P), INVALID), (dict(weight_decay=-1.0), INVALID),
    (dict(weight_decay=NAN), INVALID),
    (dict(step=P + 4), ALIGN), (dict(norm=P + 2), ALIGN), (dict(lr_dev=P + 1), ALIGN), (dict(ws=P + 8), ALIGN),
    (dict(param=P + 2), ALIGN), (dict(grad=P + 1), ALIGN), (dict(bits=32, m=P + 1), ALIGN), (dict(m_scale=P + 2), ALIGN),
    (dict(master=P + 2, param_dtype=0), ALIGN),
])
def test_adamw(lib, kw, want):
    t = _Tensor(*_args(TENSOR, {k: v for k, v in kw.items() if k in TENSOR}))
    assert lib.fp8g_adamw((_Tensor * 1)(t), 1, *_args(ADAM, {k: v for k, v in kw.items() if k in ADAM})) == want
    assert lib.fp8g_adamw(None, 1, *ADAM.values()) == INVALID
    assert lib.fp8g_adamw((_Tensor * 1)(t), -1, *ADAM.values()) == INVALID


# ------------------------------------------------------------------ the binding (CPU tensors: refused before the library)

def _f32(*shape):
    return torch.zeros(shape)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


I32 = torch.int32


@pytest.mark.parametrize("call", [
    lambda: g.moe_route(_f32(4), 2),
    lambda: g.moe_route(torch.zeros(4, 8, dtype=torch.float16), 2),
    lambda: g.moe_route(_f32(4, 8), 2, score="tanh"),
    lambda: g.moe_route(_f32(4, 8), 2, bias=_bf16(8)),
    lambda: g.moe_route(_f32(4, 8), 2, bias=_f32(7)),
    lambda: g.moe_route(_f32(4, 8), 2, token_mask=torch.ones(3, dtype=torch.bool)),
    lambda: g.moe_route(_f32(4, 8), 2),  # not on a GPU
    lambda: g.moe_route_backward(_f32(4, 8), torch.zeros(3, 2, dtype=I32), _f32(4, 2)),
    lambda: g.moe_route_backward(_f32(4, 8), torch.zeros(4, 2, dtype=torch.int64), _f32(4, 2)),
    lambda: g.residual_rms_norm(_f32(4, 8), _f32(4, 9), _f32(8)),
    lambda: g.residual_rms_norm(_f32(4, 8), _f32(4, 8), _f32(7)),
    lambda: g.residual_rms_norm(_f32(4, 8), _f32(4, 8), _f32(8), gate=_bf16(8)),
    lambda: g.residual_rms_norm(_f32(4, 8), _f32(4, 8), _f32(8), out_dtype=torch.bfloat16),
    lambda: g.residual_rms_norm(_f32(8, 4).t(), None, _f32(8)),
    lambda: g.residual_rms_norm(_f32(4, 8), None, _f32(8)),
    lambda: g.residual_rms_norm_backward(_f32(4, 8), None, None, None, _f32(4)),
    lambda: g.residual_rms_norm_backward(_f32(4, 8), _bf16(4, 8), _f32(4, 8), None, _f32(4)),
    lambda: g.residual_rms_norm_backward(_f32(4, 8), None, _f32(4, 8), None, _f32(5)),
    lambda: g.swiglu(_f32(4, 16)),
    lambda: g.swiglu(_bf16(4, 15)),
    lambda: g.swiglu(_bf16(4, 16)),
    lambda: g.fp8_swiglu_quantize_1x128(_bf16(4, 256), torch.zeros(4, 128, dtype=torch.uint8), _f32(1, 3)),
    lambda: g.fp8_swiglu_quantize_1x128(_bf16(4, 256), torch.zeros(4, 64, dtype=torch.uint8), _f32(1, 4)),
    lambda: g.fp8_swiglu_quantize_1x128(_bf16(4, 256), h=_bf16(3, 128)),
    lambda: g.fp8_swiglu_quantize_1x128_masked(_bf16(4, 256), torch.zeros(4, 128, dtype=torch.uint8), _f32(1, 4),
                                               torch.zeros(4, dtype=I32)),
    lambda: g.fp8_swiglu_quantize_1x128_masked(_bf16(2, 4, 256), torch.zeros(2, 4, 128, dtype=torch.uint8), _f32(1, 8),
                                               torch.zeros(3, dtype=I32)),
    lambda: g.swiglu_backward(_bf16(4, 16), _bf16(4, 16)),
    lambda: g.swiglu_backward(_bf16(3, 8), _bf16(4, 16)),
    lambda: g.AdamWList([], []),
    lambda: g.AdamWList([_f32(8)], []),
    lambda: g.AdamWList([_f32(8)], [_f32(7)]),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], state_bits=16),
    lambda: g.AdamWList([_f32(8, 8).t()], [_f32(8, 8)]),
    lambda: g.AdamWList([torch.zeros(8, dtype=torch.float16)], [_f32(8)]),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], weight_decay=[0.1, 0.1]),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], weight_decay=-0.1),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], masters=[_f32(8)]),
    lambda: g.AdamWList([_bf16(8)], [_f32(8)], masters=[_f32(7)]),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], m=[_f32(7)]),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], m_scales=[_f32(1)]),
    lambda: g.AdamWList([_f32(8)], [_f32(8)], step=_f32(1)),
    lambda: g.AdamWList([_f32(8)], [_f32(8)]),  # not on a GPU
])
def test_binding_refuses(call):
    with pytest.raises(ValueError):
        call()
