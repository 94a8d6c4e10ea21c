"""Training operators of whole MoE blocks: the router with sigmoid or softmax scores, balance bias and expert groups; the
RMS norms around a block with its gate and residual; the gated activation between an expert's two grouped GEMMs,
quantised for the second; each with its gradient; and the AdamW step over many tensors.

The ``fp8g_*`` and ``fp8_*`` functions carry the C ABI's names (declared, with their formulas, in
``include/fp8gemm.h``) and write into the caller's tensors; the ones without the prefix allocate their results with torch
and call those:

    ids, w, counts = moe_route(logits, topk, bias, groups=8, topk_groups=4)
    dlogits = moe_route_backward(logits, ids, dw)
    h, y, rstd, rstd_f = residual_rms_norm(x, f, weight, gate=gate, scale=0.5, post_norm=True, post_weight=post)
    dx, df, dweight, dgate, dpost = residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, weight, gate=gate, ...)
    q, sA, a = swiglu_quantize_1x128(gu, keep=True)
    dgu, a = swiglu_backward(da, gu)
    opt = AdamWList(params, grads, state_bits=8)
    adamw_step(opt, lr, norm=grad_norm(grads), max_norm=1.0)

Work is enqueued on the current CUDA stream of the tensors' device, which has to be the current device; nothing
synchronises (but the making of an ``AdamWList``, which fills its states).
"""

from __future__ import annotations

import ctypes

import torch

from . import _is_fp8, lib
from .block_ops import (_DTYPES, _F32, _I32, _U8, _all_at, _dtype, _empty, _mask, _on, _one_device, _opt, _raise, _refuse,
                        _rows, _scratch, _vector, _workspace)

_BF16 = torch.bfloat16
_SCORES = {"sigmoid": 0, "softmax": 1}


# ------------------------------------------------------------------ router

def _score(score: str) -> int:
    code = _SCORES.get(score)
    if code is None:
        _refuse("score: 'sigmoid' or 'softmax'")
    return code


def fp8g_moe_route(logits, topk: int, topk_ids, topk_weights, counts, bias=None, score: str = "sigmoid", groups: int = 1,
                   topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, token_mask=None) -> None:
    """logits [T,E] bf16 or f32, bias f32 [E] or None -> topk_ids int32 [T,topk], topk_weights f32 [T,topk], counts
    int32 [E].  token_mask: bool or uint8 [T], False for padding tokens."""
    if logits.dim() != 2:
        _refuse("logits: [T,E]")
    T, E = logits.shape
    _vector(topk_ids, T * topk, _I32, "topk_ids")
    _vector(topk_weights, T * topk, _F32, "topk_weights")
    _vector(counts, E, _I32, "counts")
    _one_device(logits.get_device(), topk_ids, topk_weights, counts)
    _route(logits, topk, topk_ids, topk_weights, counts, bias, score, groups, topk_groups, renormalize, scale, token_mask)


def _route(logits, topk, ids, weights, counts, bias, score, groups, topk_groups, renormalize, scale, token_mask) -> None:
    """The inputs' checks and the call."""
    code, ld = _dtype(logits, "logits"), _rows(logits, "logits")
    T, E = logits.shape
    if bias is not None:
        _vector(bias, E, _F32, "bias")
    mask = None if token_mask is None else _mask(token_mask, T)
    dev = logits.get_device()
    _one_device(dev, bias, token_mask)
    st = lib().fp8g_moe_route(logits.data_ptr(), code, T, E, ld, topk, _opt(bias), _score(score), groups, topk_groups,
                              1 if renormalize else 0, scale, mask, ids.data_ptr(), weights.data_ptr(),
                              counts.data_ptr(), _on(logits, dev))
    if st:
        _raise(st, "fp8g_moe_route")


def moe_route(logits, topk: int, bias=None, score: str = "sigmoid", groups: int = 1, topk_groups: int = 1,
              renormalize: bool = True, scale: float = 1.0, token_mask=None):
    """logits [T,E] -> (topk_ids int32 [T,topk], topk_weights f32 [T,topk], counts int32 [E])."""
    if logits.dim() != 2:
        _refuse("logits: [T,E]")
    T, E = logits.shape
    dev = logits.device
    ids = _empty((T, topk), dtype=_I32, device=dev)
    w = _empty((T, topk), dtype=_F32, device=dev)
    counts = _empty(E, dtype=_I32, device=dev)
    _route(logits, topk, ids, w, counts, bias, score, groups, topk_groups, renormalize, scale, token_mask)
    return ids, w, counts


def fp8g_moe_route_backward(logits, topk_ids, dweights, dlogits, score: str = "sigmoid", renormalize: bool = True,
                            scale: float = 1.0, token_mask=None) -> None:
    """topk_ids int32 [T,topk], dweights f32 [T,topk] -> dlogits [T,E] of logits' type."""
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
        _refuse("dlogits: logits' shape and type")
    code, ld, ldd = _dtype(logits, "logits"), _rows(logits, "logits"), _rows(dlogits, "dlogits")
    T, E = logits.shape
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        _refuse("topk_ids: int32 [T,topk]")
    topk = topk_ids.shape[1]
    _vector(topk_ids, T * topk, _I32, "topk_ids")
    _vector(dweights, T * topk, _F32, "dweights")
    mask = None if token_mask is None else _mask(token_mask, T)
    dev = logits.get_device()
    _one_device(dev, topk_ids, dweights, dlogits, token_mask)
    st = lib().fp8g_moe_route_backward(logits.data_ptr(), code, T, E, ld, topk, _score(score), 1 if renormalize else 0,
                                       scale, mask, topk_ids.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(), ldd,
                                       _on(logits, dev))
    if st:
        _raise(st, "fp8g_moe_route_backward")


def moe_route_backward(logits, topk_ids, dweights, score: str = "sigmoid", renormalize: bool = True, scale: float = 1.0,
                       token_mask=None):
    """The gradient of moe_route's weights with respect to the logits -> dlogits [T,E]."""
    dlogits = _empty(logits.shape, dtype=logits.dtype, device=logits.device)
    fp8g_moe_route_backward(logits, topk_ids, dweights, dlogits, score, renormalize, scale, token_mask)
    return dlogits


# ------------------------------------------------------------------ norms around a block

def _weights(n: int, weight, post_weight, gate) -> int:
    """The common type of the weights that are there (f32 where none is)."""
    code = None
    for t in (weight, post_weight, gate):
        if t is not None:
            c = _dtype(t, "weight, post_weight, gate")
            if t.numel() != n or not t.is_contiguous():
                _refuse(f"weight, post_weight, gate: [{n}], contiguous")
            if code is not None and c != code:
                _refuse("weight, post_weight and gate: one type")
            code = c
    return 1 if code is None else code


def _like(t, shape, dtype, what: str) -> int:
    """The row stride of a matrix of that shape and type."""
    if t.shape != shape or t.dtype != dtype:
        _refuse(f"{what}: {dtype} [{shape[0]},{shape[1]}]")
    return _rows(t, what)


def fp8g_residual_rms_norm(x, f, weight, h, y, rstd=None, rstd_f=None, gate=None, scale: float = 1.0,
                           post_norm: bool = False, post_weight=None, eps: float = 1e-6) -> None:
    """x [M,N] and f [M,N] (or None) -> h [M,N] of x's type (or None), y [M,N] of f's type (or None), rstd and rstd_f
    f32 [M] (or None); weight, gate, post_weight [N] or None.  h may be x."""
    shape, block = x.shape, x.dtype
    if y is not None:
        block = y.dtype
    elif f is not None:
        block = f.dtype
    ldy = 0 if y is None else _like(y, shape, block, "y")
    ldh = 0 if h is None else _like(h, shape, x.dtype, "h")
    if rstd is not None:
        _vector(rstd, shape[0], _F32, "rstd")
    if rstd_f is not None:
        _vector(rstd_f, shape[0], _F32, "rstd_f")
    _one_device(x.get_device(), h, y, rstd, rstd_f)
    _residual(x, f, block, weight, gate, scale, post_norm, post_weight, eps, _opt(h), ldh, _opt(y), ldy, _opt(rstd_f),
              _opt(rstd))


def _residual(x, f, block, weight, gate, scale, post_norm, post_weight, eps, h, ldh, y, ldy, rstd_f, rstd) -> None:
    """The inputs' checks and the call."""
    xd, ldx = _dtype(x, "x"), _rows(x, "x")
    M, N = shape = x.shape
    ldf, ptr_f = 0, None
    if f is not None:
        ldf, ptr_f = _like(f, shape, block, "f"), f.data_ptr()
    bd = _DTYPES.get(block)
    if bd is None:
        _refuse("f, y: bf16 or f32")
    wd = _weights(N, weight, post_weight, gate)
    dev = x.get_device()
    _one_device(dev, f, weight, post_weight, gate)
    st = lib().fp8g_residual_rms_norm(x.data_ptr(), ldx, ptr_f, ldf, xd, bd, M, N, 1 if post_norm else 0,
                                      _opt(post_weight), _opt(gate), scale, _opt(weight), wd, eps, h, ldh, y, ldy, rstd_f,
                                      rstd, _on(x, dev))
    if st:
        _raise(st, "fp8g_residual_rms_norm")


def residual_rms_norm(x, f=None, weight=None, gate=None, scale: float = 1.0, post_norm: bool = False, post_weight=None,
                      eps: float = 1e-6, out_dtype=None):
    """x [M,N], f [M,N] or None -> (h [M,N] of x's type, y [M,N] of f's type (without f: out_dtype, or x's), rstd f32 [M],
    rstd_f f32 [M]).  Without f h is x; without post_norm rstd_f is None."""
    dev, shape = x.device, x.shape
    if len(shape) != 2:
        _refuse("x: 2-D, rows contiguous")
    block = out_dtype or x.dtype
    h, ptr_h, rstd_f = x, None, None
    if f is not None:
        block = f.dtype
        if out_dtype not in (None, block):
            _refuse("out_dtype: f's type")
        h = _empty(shape, dtype=x.dtype, device=dev)
        ptr_h = h.data_ptr()
    y = _empty(shape, dtype=block, device=dev)
    rstd = _empty(shape[0], dtype=_F32, device=dev)
    if post_norm:
        rstd_f = _empty(shape[0], dtype=_F32, device=dev)
    N = shape[-1]
    _residual(x, f, block, weight, gate, scale, post_norm, post_weight, eps, ptr_h, N, y.data_ptr(), N, _opt(rstd_f),
              rstd.data_ptr())
    return h, y, rstd, rstd_f


def fp8g_residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, weight, dx, df=None, dweight=None, dgate=None, dpost=None,
                                    gate=None, scale: float = 1.0, post_norm: bool = False, post_weight=None,
                                    workspace=None) -> None:
    """dy [M,N] (or None), dh [M,N] of h's type (or None), h and f as the forward call had them -> dx [M,N] of h's type,
    df [M,N] of f's type (None where there was no f), dweight, dgate, dpost f32 [N] (or None).  workspace: a uint8 tensor
    of fp8g_residual_rms_norm_backward_workspace bytes (allocated if None)."""
    xd, lddx = _dtype(dx, "dx"), _rows(dx, "dx")
    M, N = shape = dx.shape
    blocks = [t for t in (dy, f, df) if t is not None]
    block = blocks[0].dtype if blocks else dx.dtype
    bd = _DTYPES.get(block)
    if bd is None:
        _refuse("dy, f, df: bf16 or f32")
    lddy, lddh, ldh, ldf, lddf = (0 if t is None else _like(t, shape, d, what) for t, d, what in (
        (dy, block, "dy"), (dh, dx.dtype, "dh"), (h, dx.dtype, "h"), (f, block, "f"), (df, block, "df")))
    wd = _weights(N, weight, post_weight, gate)
    for t, n, what in ((rstd, M, "rstd"), (rstd_f, M, "rstd_f"), (dweight, N, "dweight"), (dgate, N, "dgate"),
                       (dpost, N, "dpost")):
        if t is not None:
            _vector(t, n, _F32, what)
    if workspace is not None:
        _scratch(workspace)
    dev = dx.get_device()
    _one_device(dev, dy, dh, h, f, df, rstd, rstd_f, weight, post_weight, gate, dweight, dgate, dpost, workspace)
    if workspace is None and (dweight is not None or dgate is not None or dpost is not None):
        workspace = _workspace("fp8g_residual_rms_norm_backward_workspace", dx.device, M, N)
    st = lib().fp8g_residual_rms_norm_backward(
        _opt(dy), lddy, _opt(dh), lddh, _opt(h), ldh, _opt(f), ldf, xd, bd, M, N, 1 if post_norm else 0,
        _opt(post_weight), _opt(gate), scale, _opt(weight), wd, _opt(rstd_f), _opt(rstd), dx.data_ptr(), lddx, _opt(df),
        lddf, _opt(dweight), _opt(dgate), _opt(dpost), _opt(workspace), 0 if workspace is None else workspace.numel(),
        _on(dx, dev))
    if st:
        _raise(st, "fp8g_residual_rms_norm_backward")


def residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f=None, weight=None, gate=None, scale: float = 1.0,
                               post_norm: bool = False, post_weight=None, weight_grads: bool = True):
    """-> (dx of h's type, df of f's type or None, dweight, dgate, dpost f32 [N]); the last three are None for weights that
    there are none of, or without weight_grads.  dh may be None (nothing else uses h)."""
    if h is None or h.dim() != 2:
        _refuse("h: as residual_rms_norm returned it")
    dev, N = h.device, h.shape[-1]

    def grad(t):
        return _empty(N, dtype=_F32, device=dev) if t is not None and weight_grads else None

    dx = _empty(h.shape, dtype=h.dtype, device=dev)
    df = None if f is None else _empty(f.shape, dtype=f.dtype, device=dev)
    dw, dgate, dpost = grad(None if dy is None else weight), grad(gate), grad(post_weight)
    fp8g_residual_rms_norm_backward(dy, dh, h, f, rstd, rstd_f, weight, dx, df, dw, dgate, dpost, gate, scale, post_norm,
                                    post_weight)
    return dx, df, dw, dgate, dpost


# ------------------------------------------------------------------ gated activation

def _bf16_rows(t, cols: int, what: str) -> int:
    if t.dtype != _BF16 or t.dim() != 2 or t.shape[1] != cols:
        _refuse(f"{what}: bf16 [M,{cols}]")
    return _rows(t, what)


def _gate_up(gu) -> int:
    if gu.dtype != _BF16 or gu.dim() not in (2, 3) or gu.shape[-1] % 2:
        _refuse("gu: bf16 [M,2F]")
    return gu.shape[-1] // 2


def fp8_swiglu_quantize_1x128(gu, q=None, sA=None, h=None) -> None:
    """gu bf16 [M,2F] -> q e4m3 [M,F] and sA f32 [F/128, ld_sa >= M], and h bf16 [M,F] (or None; q may be None too)."""
    F = _gate_up(gu)
    ldgu = _bf16_rows(gu, 2 * F, "gu")
    M = gu.shape[0]
    ldq = ldh = ld_sa = 0
    if q is not None:
        if not _is_fp8(q) or q.shape != (M, F):
            _refuse("q: e4m3 [M,F]")
        ldq = _rows(q, "q")
        if sA is None or sA.dtype != _F32 or sA.dim() != 2 or sA.shape[0] != F // 128 or sA.shape[1] < M or \
                (sA.stride(1) != 1 and sA.shape[1] > 1):
            _refuse("sA: f32 [F/128, ld_sa >= M]")
        ld_sa = sA.stride(0) if sA.shape[0] > 1 else sA.shape[1]
    if h is not None:
        ldh = _bf16_rows(h, F, "h")
        if h.shape[0] != M:
            _refuse("h: bf16 [M,F]")
    dev = gu.get_device()
    _one_device(dev, q, sA, h)
    st = lib().fp8_swiglu_quantize_1x128(gu.data_ptr(), M, F, ldgu, _opt(q), ldq, _opt(sA), ld_sa, _opt(h), ldh,
                                         _on(gu, dev))
    if st:
        _raise(st, "fp8_swiglu_quantize_1x128")


def fp8_swiglu_quantize_1x128_masked(gu, q, sA, masked_m) -> None:
    """gu bf16 [E,cap,2F] -> q e4m3 [E,cap,F], sA f32 [F/128, ld_sa >= E*cap]: only rows m < masked_m[e]."""
    F = _gate_up(gu)
    if gu.dim() != 3 or not gu.is_contiguous():
        _refuse("gu: bf16 [E,cap,2F] contiguous")
    E, cap = gu.shape[:2]
    if not _is_fp8(q) or q.shape != (E, cap, F) or not q.is_contiguous():
        _refuse("q: e4m3 [E,cap,F] contiguous")
    if sA.dtype != _F32 or sA.dim() != 2 or sA.shape[0] != F // 128 or sA.shape[1] < E * cap or \
            (sA.stride(1) != 1 and sA.shape[1] > 1):
        _refuse("sA: f32 [F/128, ld_sa >= E*cap]")
    _vector(masked_m, E, _I32, "masked_m")
    dev = gu.get_device()
    _one_device(dev, q, sA, masked_m)
    st = lib().fp8_swiglu_quantize_1x128_masked(gu.data_ptr(), E, cap, F, masked_m.data_ptr(), q.data_ptr(),
                                                sA.data_ptr(), sA.stride(0) if sA.shape[0] > 1 else sA.shape[1],
                                                _on(gu, dev))
    if st:
        _raise(st, "fp8_swiglu_quantize_1x128_masked")


def swiglu_quantize_1x128(gu, ld_sa: int | None = None, keep: bool = False):
    """bf16 [M,2F] -> (q uint8 [M,F], sA f32 [F/128, ld_sa], h bf16 [M,F] with keep, else None); ld_sa defaults to M rounded
    up to 4.  (Columns of sA past M are not written.)"""
    F = _gate_up(gu)
    M, dev = gu.shape[0], gu.device
    q = _empty((M, F), dtype=_U8, device=dev)
    sA = _empty((F // 128, ld_sa or max((M + 3) // 4 * 4, 4)), dtype=_F32, device=dev)
    h = _empty((M, F), dtype=_BF16, device=dev) if keep else None
    fp8_swiglu_quantize_1x128(gu, q, sA, h)
    return q, sA, h


def swiglu(gu):
    """bf16 [M,2F] -> h bf16 [M,F], not quantised."""
    F = _gate_up(gu)
    h = _empty((gu.shape[0], F), dtype=_BF16, device=gu.device)
    fp8_swiglu_quantize_1x128(gu, h=h)
    return h


def fp8g_swiglu_backward(dh, gu, dgu, h=None) -> None:
    """dh bf16 [M,F], gu bf16 [M,2F] -> dgu bf16 [M,2F] (may be gu itself), h bf16 [M,F] (or None)."""
    F = _gate_up(gu)
    ldgu, lddgu, lddh = _bf16_rows(gu, 2 * F, "gu"), _bf16_rows(dgu, 2 * F, "dgu"), _bf16_rows(dh, F, "dh")
    M = gu.shape[0]
    if dgu.shape[0] != M or dh.shape[0] != M or (h is not None and h.shape[0] != M):
        _refuse("dh, dgu, h: gu's rows")
    ldh = 0 if h is None else _bf16_rows(h, F, "h")
    dev = gu.get_device()
    _one_device(dev, dh, dgu, h)
    st = lib().fp8g_swiglu_backward(dh.data_ptr(), lddh, gu.data_ptr(), M, F, ldgu, dgu.data_ptr(), lddgu, _opt(h), ldh,
                                    _on(gu, dev))
    if st:
        _raise(st, "fp8g_swiglu_backward")


def swiglu_backward(dh, gu, keep: bool = True):
    """-> (dgu bf16 [M,2F], h bf16 [M,F] with keep, else None: what the second product's weight gradient needs)."""
    F = _gate_up(gu)
    dgu = _empty(gu.shape, dtype=_BF16, device=gu.device)
    h = _empty((gu.shape[0], F), dtype=_BF16, device=gu.device) if keep else None
    fp8g_swiglu_backward(dh, gu, dgu, h)
    return dgu, h


# ------------------------------------------------------------------ AdamW

class _Tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_WORKSPACE = 64  # FP8G_ADAMW_WORKSPACE


class AdamWList:
    """The parameters of a program with their gradients and AdamW states, checked and listed once.

    params: bf16 or f32, grads: bf16 or f32 of the same shapes, all contiguous.  masters: True for fp32 copies of the bf16
    parameters, made here, or a sequence of f32 tensors (None for an f32 parameter).  state_bits 32: states m and v in
    f32; 8: e4m3 codes (uint8) of m and of v's root, with m_scales and v_scales (f32, one for each 128 values).
    weight_decay: a number, or one for each parameter.  m, v, m_scales, v_scales, step: the states of a run that goes on
    (step int64 [1] on the device: the steps taken); zeros if None.

    It holds the tensors and the memory that they had, so nothing else comes to lie there.  A call refuses a list whose
    tensors have been given other memory since: a program whose tensors move makes a new one.  Results that overlap are
    refused here."""

    def __init__(self, params, grads, masters=None, state_bits: int = 32, weight_decay=0.01, m=None, v=None,
                 m_scales=None, v_scales=None, step=None):
        self.params, self.grads = params, grads = list(params), list(grads)
        self.n = n = len(params)
        if n == 0 or len(grads) != n:
            _refuse("params, grads: at least one tensor, a gradient for each")
        if state_bits not in (8, 32):
            _refuse("state_bits: 8 or 32")
        self.state_bits = state_bits
        self.device, self.device_index = params[0].device, params[0].get_device()
        for p, d in zip(params, grads):
            _dtype(p, "params")
            _dtype(d, "grads")
            if p.shape != d.shape or not p.is_contiguous() or not d.is_contiguous():
                _refuse("params, grads: the same shapes, contiguous")
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(w) for w in weight_decay]
        if len(decay) != n or not all(w >= 0.0 for w in decay):
            _refuse("weight_decay: >= 0, a number or one for each parameter")
        sizes = [p.numel() for p in params]
        if masters is True:
            masters = [p.detach().float() if p.dtype == _BF16 else None for p in params]
        self.masters = masters = [None] * n if masters is None or masters is False else list(masters)
        code, blocks = (_F32, None) if state_bits == 32 else (_U8, [(s + 127) // 128 for s in sizes])
        self.m, self.v = self._states(m, sizes, code, "m"), self._states(v, sizes, code, "v")
        if state_bits == 8:
            self.m_scales = self._states(m_scales, blocks, _F32, "m_scales")
            self.v_scales = self._states(v_scales, blocks, _F32, "v_scales")
        else:
            if m_scales is not None or v_scales is not None:
                _refuse("m_scales, v_scales: with state_bits 8")
            self.m_scales = self.v_scales = [None] * n
        if step is None:
            step = torch.zeros(1, dtype=torch.int64, device=self.device)
        _vector(step, 1, torch.int64, "step")
        self.step = step
        if len(masters) != n:
            _refuse("masters: one for each parameter (None for f32)")
        for p, t in zip(params, masters):
            if t is not None:
                if p.dtype != _BF16:
                    _refuse("masters: of bf16 parameters")
                _vector(t, p.numel(), _F32, "masters")
        written = [t for ts in (params, masters, self.m, self.v, self.m_scales, self.v_scales) for t in ts if t is not None]
        self.tensors = tensors = written + grads
        _one_device(self.device_index, step, *tensors)
        self.places = [t.data_ptr() for t in tensors]
        self.memory = [t.untyped_storage() for t in tensors]
        self.indices = list(range(len(tensors)))
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i < len(written))
                       for i, t in enumerate(tensors) if t.numel())
        end = known = 0  # of what is written, and of all
        for at, to, result in spans:
            if at < end or (result and at < known):
                _refuse("params, states: one overlaps another tensor of the list")
            known = max(known, to)
            end = max(end, to) if result else end
        self.table = (_Tensor * n)(*[
            _Tensor(p.data_ptr(), d.data_ptr(), a.data_ptr(), b.data_ptr(), _opt(sa), _opt(sb), _opt(t), p.numel(), w,
                    _DTYPES[p.dtype], _DTYPES[d.dtype], 0)
            for p, d, a, b, sa, sb, t, w in zip(params, grads, self.m, self.v, self.m_scales, self.v_scales, masters, decay)])
        self.workspace = _empty(_WORKSPACE, dtype=_U8, device=self.device)

    def _states(self, given, sizes, dtype, what: str):
        """The given states, or zeros: views of one buffer, each from a multiple of 128 values on."""
        if given is None:
            starts = [0]
            for s in sizes:
                starts.append(starts[-1] + (s + 127) // 128 * 128)
            flat = torch.zeros(starts[-1], dtype=dtype, device=self.device)
            return [flat[a: a + s] for a, s in zip(starts, sizes)]
        given = list(given)
        if len(given) != len(sizes):
            _refuse(f"{what}: one for each parameter")
        for t, s in zip(given, sizes):
            if not (dtype == _U8 and t.dtype == torch.float8_e4m3fn):
                _vector(t, s, dtype, what)
            elif t.numel() != s or not t.is_contiguous():
                _refuse(f"{what}: [{s}], contiguous")
        return given

    def __len__(self):
        return self.n

    def check_places(self) -> None:
        """Every tensor where it was when it was listed."""
        if not _all_at(self.tensors, self.places, self.indices):
            _refuse("params, grads: a tensor has moved since it was listed")


def adamw_step(tensors: AdamWList, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, norm=None,
               max_norm: float | None = None, norm_eps: float = 1e-6) -> None:
    """One AdamW step, in place.  lr: a number, or an f32 [1] tensor on the device (for a captured graph).  norm: f32 [1] as
    grad_norm returned it; with it the gradients are taken times min(1, max_norm / (norm + norm_eps)) (max_norm None: as they
    are), and the step is left out where it is not finite."""
    fp8g_adamw(tensors, lr, beta1, beta2, eps, norm, max_norm, norm_eps)


def fp8g_adamw(tensors: AdamWList, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, norm=None,
               max_norm: float | None = None, norm_eps: float = 1e-6, workspace=None) -> None:
    """adamw_step; workspace: a uint8 tensor of FP8G_ADAMW_WORKSPACE bytes (the list's own if None)."""
    tensors.check_places()
    dev = tensors.device_index
    lr_dev = None
    if isinstance(lr, torch.Tensor):
        _vector(lr, 1, _F32, "lr")
        _one_device(dev, lr)
        lr, lr_dev = 0.0, lr.data_ptr()
    if norm is not None:
        _vector(norm, 1, _F32, "norm")
        _one_device(dev, norm)
    ws = tensors.workspace
    if workspace is not None:
        _scratch(workspace)
        _one_device(dev, workspace)
        ws = workspace
    st = lib().fp8g_adamw(tensors.table, tensors.n, tensors.state_bits, lr, lr_dev, beta1, beta2, eps,
                          tensors.step.data_ptr(), _opt(norm), float("inf") if max_norm is None else max_norm, norm_eps,
                          ws.data_ptr(), ws.numel(), _on(ws, dev))
    if st:
        _raise(st, "fp8g_adamw")
