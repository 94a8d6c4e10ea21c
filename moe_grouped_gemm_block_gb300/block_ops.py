"""Training operators around the grouped GEMMs: layer norm, the MoE gate with its balance loss, the combine of
the experts' rows, each with its gradient, and the global gradient norm with clipping.

The ``fp8g_*`` functions carry the C ABI's names (declared, with their formulas, in ``include/fp8gemm.h``) and write
into the caller's tensors; the ones without the prefix allocate their results with torch and call those:

    y, mean, rstd = layer_norm(x, weight, bias)
    dx, dweight, dbias = layer_norm_backward(dy, x, weight, mean, rstd)
    ids, w, counts, loss = moe_gate(logits, topk)
    dlogits = moe_gate_backward(logits, ids, counts, dw, dloss)
    out = moe_combine(D, entry_row, w, residual=x)
    dD, dw = moe_combine_backward(dout, D, entry_row, row_token, w)
    norm = clip_grad_norm(grads, max_norm)
    norm = grad_norm(grads)

Work is enqueued on the current CUDA stream of the tensors' device; nothing synchronises.
"""

from __future__ import annotations

import ctypes

import torch

from . import _check, _need, _on_one_device, _ptr, _stream, lib

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_F32 = torch.float32
_I32 = torch.int32


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    _need(code is not None, f"{what}: bf16 or f32")
    return code


def _rows(t: torch.Tensor, what: str) -> int:
    """The row stride of a matrix whose rows are contiguous."""
    _need(t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1), f"{what}: 2-D, rows contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _opt(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _vector(t: torch.Tensor | None, n: int, dtype, what: str) -> None:
    _need(t is None or (t.dtype == dtype and t.numel() == n and t.is_contiguous()),
          f"{what}: {dtype} [{n}], contiguous")


def _workspace(name: str, device, *sizes) -> torch.Tensor:
    n = ctypes.c_int64()
    _check(getattr(lib(), name)(*sizes, ctypes.byref(n)), name)
    return torch.empty(max(n.value, 16), dtype=torch.uint8, device=device)


def _scratch(t: torch.Tensor) -> torch.Tensor:
    _need(t.dtype == torch.uint8 and t.is_contiguous(), "workspace: uint8, contiguous")
    return t


# ------------------------------------------------------------------ layer norm

def _norm_weights(weight, bias, n: int) -> int:
    code = 1
    for t, what in ((bias, "bias"), (weight, "weight")):
        if t is not None:
            code = _dtype(t, what)
            _need(t.numel() == n and t.is_contiguous(), f"{what}: [{n}], contiguous")
    _need(weight is None or bias is None or weight.dtype == bias.dtype, "weight and bias: one type")
    return code


def fp8g_layer_norm(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5) -> None:
    """x [M,N] -> y [M,N] (bf16 or f32 each), mean and rstd f32 [M] (or None); weight, bias [N] or None."""
    xd, yd, ldx, ldy = _dtype(x, "x"), _dtype(y, "y"), _rows(x, "x"), _rows(y, "y")
    M, N = x.shape
    _need(y.shape == x.shape, "y: x's shape")
    wd = _norm_weights(weight, bias, N)
    _vector(mean, M, _F32, "mean")
    _vector(rstd, M, _F32, "rstd")
    _on_one_device(x, *(t for t in (weight, bias, y, mean, rstd) if t is not None))
    _check(lib().fp8g_layer_norm(_ptr(x), xd, M, N, ldx, _opt(weight), _opt(bias), wd, eps, _ptr(y), yd, ldy,
                                 _opt(mean), _opt(rstd), _stream(x)), "fp8g_layer_norm")


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out_dtype=None):
    """x [M,N] bf16 or f32 -> (y [M,N] of out_dtype (x's), mean f32 [M], rstd f32 [M])."""
    y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    mean = torch.empty(x.shape[0], dtype=_F32, device=x.device)
    rstd = torch.empty(x.shape[0], dtype=_F32, device=x.device)
    fp8g_layer_norm(x, weight, bias, y, mean, rstd, eps)
    return y, mean, rstd


def fp8g_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, workspace=None) -> None:
    """dy [M,N], x [M,N], weight [N] or None, mean and rstd f32 [M] -> dx [M,N] of x's type, dweight and dbias f32 [N]
    (or None).  workspace: a uint8 tensor of fp8g_layer_norm_backward_workspace bytes (allocated if None)."""
    yd, xd = _dtype(dy, "dy"), _dtype(x, "x")
    lddy, ldx, lddx = _rows(dy, "dy"), _rows(x, "x"), _rows(dx, "dx")
    M, N = x.shape
    _need(dy.shape == x.shape and dx.shape == x.shape and dx.dtype == x.dtype, "dy, dx: x's shape; dx: x's type")
    wd = _norm_weights(weight, None, N)
    for t, n, what in ((mean, M, "mean"), (rstd, M, "rstd"), (dweight, N, "dweight"), (dbias, N, "dbias")):
        _vector(t, n, _F32, what)
    _need(mean is not None and rstd is not None, "mean, rstd: as layer_norm returned them")
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = _workspace("fp8g_layer_norm_backward_workspace", x.device, M, N)
    if workspace is not None:
        _scratch(workspace)
    _on_one_device(x, *(t for t in (dy, weight, mean, rstd, dx, dweight, dbias, workspace) if t is not None))
    _check(lib().fp8g_layer_norm_backward(_ptr(dy), yd, lddy, _ptr(x), xd, ldx, _opt(weight), wd, _ptr(mean),
                                          _ptr(rstd), M, N, _ptr(dx), lddx, _opt(dweight), _opt(dbias),
                                          _opt(workspace), 0 if workspace is None else workspace.numel(),
                                          _stream(x)), "fp8g_layer_norm_backward")


def layer_norm_backward(dy, x, weight, mean, rstd, weight_grads: bool = True):
    """-> (dx of x's type, dweight f32 [N], dbias f32 [N]); the last two are None without weight_grads."""
    N = x.shape[1]
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty(N, dtype=_F32, device=x.device) if weight_grads else None
    db = torch.empty(N, dtype=_F32, device=x.device) if weight_grads else None
    fp8g_layer_norm_backward(dy, x, weight, mean, rstd, dx, dw, db)
    return dx, dw, db


# ------------------------------------------------------------------ gate

def _mask(mask, T: int):
    _need(mask is None or (mask.dtype in (torch.bool, torch.uint8) and mask.numel() == T and mask.is_contiguous()),
          f"token_mask: bool or uint8 [{T}], contiguous")
    return mask


def fp8g_moe_gate(logits, topk: int, topk_ids, topk_weights, counts, loss=None, renormalize: bool = True,
                  loss_coef: float = 0.01, token_mask=None, workspace=None) -> None:
    """logits [T,E] bf16 or f32 -> topk_ids int32 [T,topk], topk_weights f32 [T,topk], counts int32 [E], loss f32 [1]
    (or None).  token_mask: bool or uint8 [T], False for padding tokens."""
    code, ld = _dtype(logits, "logits"), _rows(logits, "logits")
    T, E = logits.shape
    _vector(topk_ids, T * topk, _I32, "topk_ids")
    _vector(topk_weights, T * topk, _F32, "topk_weights")
    _vector(counts, E, _I32, "counts")
    _vector(loss, 1, _F32, "loss")
    _mask(token_mask, T)
    if workspace is None:
        workspace = _workspace("fp8g_moe_gate_workspace", logits.device, T, E)
    _scratch(workspace)
    _on_one_device(logits, *(t for t in (topk_ids, topk_weights, counts, loss, token_mask, workspace) if t is not None))
    _check(lib().fp8g_moe_gate(_ptr(logits), code, T, E, ld, topk, int(renormalize), _opt(token_mask), loss_coef,
                               _ptr(topk_ids), _ptr(topk_weights), _ptr(counts), _opt(loss), _ptr(workspace),
                               workspace.numel(), _stream(logits)), "fp8g_moe_gate")


def moe_gate(logits, topk: int, renormalize: bool = True, loss_coef: float = 0.01, token_mask=None):
    """logits [T,E] -> (topk_ids int32 [T,topk], topk_weights f32 [T,topk], counts int32 [E], balance loss f32 [1])."""
    _need(logits.dim() == 2, "logits: [T,E]")
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, topk), dtype=_I32, device=dev)
    w = torch.empty((T, topk), dtype=_F32, device=dev)
    counts = torch.empty(E, dtype=_I32, device=dev)
    loss = torch.empty(1, dtype=_F32, device=dev)
    fp8g_moe_gate(logits, topk, ids, w, counts, loss, renormalize, loss_coef, token_mask)
    return ids, w, counts, loss


def fp8g_moe_gate_backward(logits, topk_ids, counts, dweights, dloss, dlogits, renormalize: bool = True,
                           loss_coef: float = 0.01, token_mask=None) -> None:
    """dweights f32 [T,topk] and dloss f32 [1] (either may be None) -> dlogits [T,E] of logits' type."""
    code, ld, ldd = _dtype(logits, "logits"), _rows(logits, "logits"), _rows(dlogits, "dlogits")
    T, E = logits.shape
    _need(dlogits.shape == logits.shape and dlogits.dtype == logits.dtype, "dlogits: logits' shape and type")
    _need(topk_ids.dim() == 2 and topk_ids.shape[0] == T, "topk_ids: int32 [T,topk]")
    topk = topk_ids.shape[1]
    _vector(topk_ids, T * topk, _I32, "topk_ids")
    _vector(counts, E, _I32, "counts")
    _vector(dweights, T * topk, _F32, "dweights")
    _vector(dloss, 1, _F32, "dloss")
    _mask(token_mask, T)
    _on_one_device(logits, *(t for t in (topk_ids, counts, dweights, dloss, dlogits, token_mask) if t is not None))
    _check(lib().fp8g_moe_gate_backward(_ptr(logits), code, T, E, ld, topk, int(renormalize), _opt(token_mask),
                                        loss_coef, _ptr(topk_ids), _ptr(counts), _opt(dweights), _opt(dloss),
                                        _ptr(dlogits), ldd, _stream(logits)), "fp8g_moe_gate_backward")


def moe_gate_backward(logits, topk_ids, counts, dweights=None, dloss=None, renormalize: bool = True,
                      loss_coef: float = 0.01, token_mask=None):
    """The gradient of moe_gate's weights and loss with respect to the logits -> dlogits [T,E]."""
    dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    fp8g_moe_gate_backward(logits, topk_ids, counts, dweights, dloss, dlogits, renormalize, loss_coef, token_mask)
    return dlogits


# ------------------------------------------------------------------ combine

def fp8g_moe_combine(D, entry_row, weights, out, residual=None) -> None:
    """D bf16 [M,N], entry_row int32 [T,topk], weights f32 [T,topk] or None (1) -> out [T,N] bf16 or f32, plus
    residual [T,N] of out's type."""
    _need(D.dtype == torch.bfloat16, "D: bf16 [M,N]")
    code, ldd, ldo = _dtype(out, "out"), _rows(D, "D"), _rows(out, "out")
    M, N = D.shape
    _need(entry_row.dim() == 2, "entry_row: int32 [T,topk]")
    T, topk = entry_row.shape
    _need(out.shape == (T, N), "out: [T,N]")
    _vector(entry_row, T * topk, _I32, "entry_row")
    _vector(weights, T * topk, _F32, "weights")
    ldr = 0
    if residual is not None:
        ldr = _rows(residual, "residual")
        _need(residual.shape == out.shape and residual.dtype == out.dtype, "residual: out's shape and type")
    _on_one_device(D, *(t for t in (entry_row, weights, out, residual) if t is not None))
    _check(lib().fp8g_moe_combine(_ptr(D), M, N, ldd, _ptr(entry_row), T, topk, _opt(weights), _opt(residual), ldr,
                                  _ptr(out), code, ldo, _stream(D)), "fp8g_moe_combine")


def moe_combine(D, entry_row, weights=None, residual=None, out_dtype=None):
    """The experts' rows D back to their tokens -> out [T,N] of out_dtype (the residual's type, or bf16)."""
    dtype = out_dtype or (D.dtype if residual is None else residual.dtype)
    out = torch.empty((entry_row.shape[0], D.shape[1]), dtype=dtype, device=D.device)
    fp8g_moe_combine(D, entry_row, weights, out, residual)
    return out


def fp8g_moe_combine_backward(dout, D, entry_row, row_token, weights, dD, dweights=None) -> None:
    """dout [T,N] bf16 or f32, D bf16 [M,N] (None if dweights is), entry_row int32 [T,topk], row_token int32 [M] ->
    dD bf16 [M,N] (padding rows zero), dweights f32 [T,topk] (or None)."""
    code, lddo, lddd = _dtype(dout, "dout"), _rows(dout, "dout"), _rows(dD, "dD")
    _need(dD.dtype == torch.bfloat16, "dD: bf16 [M,N]")
    M, N = dD.shape
    _need(entry_row.dim() == 2, "entry_row: int32 [T,topk]")
    T, topk = entry_row.shape
    _need(dout.shape == (T, N), "dout: [T,N]")
    _need(dweights is None or D is not None, "D: needed for dweights")
    ldd = 0
    if D is not None:
        ldd = _rows(D, "D")
        _need(D.dtype == torch.bfloat16 and D.shape == dD.shape, "D: bf16 [M,N]")
    _vector(entry_row, T * topk, _I32, "entry_row")
    _vector(row_token, M, _I32, "row_token")
    _vector(weights, T * topk, _F32, "weights")
    _vector(dweights, T * topk, _F32, "dweights")
    _on_one_device(dout, *(t for t in (D, entry_row, row_token, weights, dD, dweights) if t is not None))
    _check(lib().fp8g_moe_combine_backward(_ptr(dout), code, lddo, _opt(D), M, N, ldd, _ptr(entry_row),
                                           _ptr(row_token), T, topk, _opt(weights), _ptr(dD), lddd, _opt(dweights),
                                           _stream(dout)), "fp8g_moe_combine_backward")


def moe_combine_backward(dout, D, entry_row, row_token, weights=None):
    """-> (dD bf16 [M,N], dweights f32 [T,topk], or None without weights)."""
    dD = torch.empty(D.shape, dtype=torch.bfloat16, device=dout.device)
    dw = None if weights is None else torch.empty(entry_row.shape, dtype=_F32, device=dout.device)
    fp8g_moe_combine_backward(dout, D, entry_row, row_token, weights, dD, dw)
    return dD, dw


# ------------------------------------------------------------------ gradient norm

class GradList:
    """The gradients of a program (and, for clipping out of place, the tensors that take the results), checked and
    listed once.  It holds the tensors, so their memory stays; a program whose gradients move makes a new one."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        n = len(self.grads)
        _need(n > 0, "grads: at least one tensor")
        _need(len(self.out) == n, "out: a tensor for each gradient")
        self.device = self.grads[0].device
        for t, o in zip(self.grads, self.out):
            _need(t.dtype in _DTYPES and t.is_contiguous(), "grads: bf16 or f32, contiguous")
            _need(o is t or (o.dtype == t.dtype and o.shape == t.shape and o.is_contiguous()),
                  "out: each gradient's shape and type, contiguous")
            _need(t.is_cuda and t.device == self.device and o.device == self.device,
                  "grads: CUDA tensors on one device")
        self.ptrs = (ctypes.c_void_p * n)(*(t.data_ptr() for t in self.grads))
        self.out_ptrs = (ctypes.c_void_p * n)(*(t.data_ptr() for t in self.out))
        self.numels = (ctypes.c_int64 * n)(*(t.numel() for t in self.grads))
        self.dtypes = (ctypes.c_int32 * n)(*(_DTYPES[t.dtype] for t in self.grads))
        b = ctypes.c_int64()
        _check(lib().fp8g_grad_norm_workspace(n, ctypes.byref(b)), "fp8g_grad_norm_workspace")
        self.workspace_bytes = b.value

    def __len__(self):
        return len(self.grads)


def _norm_buffers(g: GradList, norm, workspace):
    _need(norm.dtype == _F32 and norm.numel() == 1, "norm: f32 [1]")
    if workspace is None:
        workspace = torch.empty(g.workspace_bytes, dtype=torch.uint8, device=g.device)
    _need(norm.device == g.device and workspace.device == g.device, "norm, workspace: on the gradients' device")
    return _scratch(workspace)


def fp8g_grad_norm(grads: GradList, norm, workspace=None) -> None:
    """norm f32 [1] = the 2-norm of all gradients together."""
    ws = _norm_buffers(grads, norm, workspace)
    _check(lib().fp8g_grad_norm(grads.ptrs, grads.numels, grads.dtypes, len(grads), _ptr(norm), _ptr(ws), ws.numel(),
                                _stream(norm)), "fp8g_grad_norm")


def fp8g_clip_grad_norm(grads: GradList, max_norm: float, norm, eps: float = 1e-6, workspace=None) -> None:
    """norm f32 [1] as fp8g_grad_norm; every gradient times min(1, max_norm / (norm + eps)), into grads.out."""
    ws = _norm_buffers(grads, norm, workspace)
    _check(lib().fp8g_clip_grad_norm(grads.ptrs, grads.out_ptrs, grads.numels, grads.dtypes, len(grads), max_norm, eps,
                                     _ptr(norm), _ptr(ws), ws.numel(), _stream(norm)), "fp8g_clip_grad_norm")


def _grad_list(grads) -> GradList:
    return grads if isinstance(grads, GradList) else GradList(grads)


def grad_norm(grads) -> torch.Tensor:
    """grads: a GradList or a sequence of tensors -> their 2-norm, f32 [1] on the device."""
    g = _grad_list(grads)
    norm = torch.empty(1, dtype=_F32, device=g.device)
    fp8g_grad_norm(g, norm)
    return norm


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + eps)), in place or, for a GradList with ``out``, into that
    -> the norm before clipping, f32 [1] on the device."""
    g = _grad_list(grads)
    norm = torch.empty(1, dtype=_F32, device=g.device)
    fp8g_clip_grad_norm(g, max_norm, norm, eps)
    return norm
