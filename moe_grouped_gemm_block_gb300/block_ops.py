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

Work is enqueued on the current CUDA stream of the tensors' device, which has to be the current device; nothing
synchronises.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import Fp8GemmError, _check, _need, _need_current, _stream, lib

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_F32 = torch.float32
_I32 = torch.int32
_U8 = torch.uint8
_empty = torch.empty

# The checks below run on every call, next to kernels of a few microseconds: they read each property of a tensor once
# and build no message unless one fails.


def _refuse(msg: str):
    raise ValueError(msg)


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        _refuse(f"{what}: bf16 or f32")
    return code


def _rows(t: torch.Tensor, what: str) -> int:
    """The row stride of a matrix whose rows are contiguous."""
    if t.dim() != 2:
        _refuse(f"{what}: 2-D, rows contiguous")
    m, n = t.shape
    ld, one = t.stride()
    if one != 1 and n != 1:
        _refuse(f"{what}: 2-D, rows contiguous")
    return ld if m > 1 else n


def _opt(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _vector(t: torch.Tensor, n: int, dtype, what: str) -> None:
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        _refuse(f"{what}: {dtype} [{n}], contiguous")


def _one_device(dev: int, *ts: torch.Tensor | None) -> None:
    """Every tensor in the memory of GPU `dev` (-1: the first one is not on a GPU)."""
    for t in ts:
        if t is not None and t.get_device() != dev:
            _refuse("operands: CUDA tensors on one device")
    if dev < 0:
        _refuse("operands: CUDA tensors on one device")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(t: torch.Tensor, dev: int) -> int:
    """The current stream of the tensor's device, which is the current one."""
    _need_current(dev)
    return _raw_stream(dev) if _raw_stream is not None else _stream(t)


def _raise(code: int, what: str):
    raise Fp8GemmError(code, what)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes) -> int:
    n = ctypes.c_int64()
    code = getattr(lib(), name)(*sizes, ctypes.byref(n))
    if code:
        _raise(code, name)
    return n.value


def _workspace(name: str, device, *sizes) -> torch.Tensor | None:
    n = _workspace_bytes(name, *sizes)
    return _empty(n, dtype=_U8, device=device) if n else None


def _scratch(t: torch.Tensor) -> None:
    if t.dtype != _U8 or not t.is_contiguous():
        _refuse("workspace: uint8, contiguous")


# ------------------------------------------------------------------ layer norm

def _norm_weights(weight, bias, n: int) -> int:
    code = 1
    for t, what in ((bias, "bias"), (weight, "weight")):
        if t is not None:
            code = _dtype(t, what)
            if t.numel() != n or not t.is_contiguous():
                _refuse(f"{what}: [{n}], contiguous")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        _refuse("weight and bias: one type")
    return code


def fp8g_layer_norm(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5) -> None:
    """x [M,N] -> y [M,N] (bf16 or f32 each), mean and rstd f32 [M] (or None); weight, bias [N] or None."""
    if y.shape != x.shape:
        _refuse("y: x's shape")
    ldy = _rows(y, "y")
    if mean is not None:
        _vector(mean, x.shape[0], _F32, "mean")
    if rstd is not None:
        _vector(rstd, x.shape[0], _F32, "rstd")
    _one_device(x.get_device(), y, mean, rstd)
    _norm(x, weight, bias, y, ldy, _opt(mean), _opt(rstd), eps)


def _norm(x, weight, bias, y, ldy: int, mean: int | None, rstd: int | None, eps: float) -> None:
    """The inputs' checks and the call."""
    xd, ldx, yd = _dtype(x, "x"), _rows(x, "x"), _dtype(y, "y")
    M, N = x.shape
    wd = 1 if weight is None and bias is None else _norm_weights(weight, bias, N)
    dev = x.get_device()
    _one_device(dev, weight, bias)
    code = lib().fp8g_layer_norm(x.data_ptr(), xd, M, N, ldx, _opt(weight), _opt(bias), wd, eps, y.data_ptr(), yd, ldy,
                                 mean, rstd, _on(x, dev))
    if code:
        _raise(code, "fp8g_layer_norm")


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out_dtype=None):
    """x [M,N] bf16 or f32 -> (y [M,N] of out_dtype (x's), mean f32 [M], rstd f32 [M])."""
    dev, shape = x.device, x.shape
    y = _empty(shape, dtype=out_dtype or x.dtype, device=dev)
    mean = _empty(shape[0], dtype=_F32, device=dev)
    rstd = _empty(shape[0], dtype=_F32, device=dev)
    _norm(x, weight, bias, y, shape[-1], mean.data_ptr(), rstd.data_ptr(), eps)
    return y, mean, rstd


def fp8g_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, workspace=None) -> None:
    """dy [M,N], x [M,N], weight [N] or None, mean and rstd f32 [M] -> dx [M,N] of x's type, dweight and dbias f32 [N]
    (or None).  workspace: a uint8 tensor of fp8g_layer_norm_backward_workspace bytes (allocated if None)."""
    if dx.shape != x.shape or dx.dtype != x.dtype:
        _refuse("dx: x's shape and type")
    lddx = _rows(dx, "dx")
    if dweight is not None:
        _vector(dweight, x.shape[1], _F32, "dweight")
    if dbias is not None:
        _vector(dbias, x.shape[1], _F32, "dbias")
    if workspace is not None:
        _scratch(workspace)
    _one_device(x.get_device(), dx, dweight, dbias, workspace)
    _norm_grad(dy, x, weight, mean, rstd, dx, lddx, dweight, dbias, workspace)


def _norm_grad(dy, x, weight, mean, rstd, dx, lddx: int, dweight, dbias, workspace) -> None:
    """The inputs' checks and the call."""
    yd, xd = _dtype(dy, "dy"), _dtype(x, "x")
    lddy, ldx = _rows(dy, "dy"), _rows(x, "x")
    M, N = shape = x.shape
    if dy.shape != shape:
        _refuse("dy: x's shape")
    wd = 1 if weight is None else _norm_weights(weight, None, N)
    if mean is None or rstd is None:
        _refuse("mean, rstd: as layer_norm returned them")
    _vector(mean, M, _F32, "mean")
    _vector(rstd, M, _F32, "rstd")
    dev = x.get_device()
    _one_device(dev, dy, weight, mean, rstd)
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = _workspace("fp8g_layer_norm_backward_workspace", x.device, M, N)
    code = lib().fp8g_layer_norm_backward(dy.data_ptr(), yd, lddy, x.data_ptr(), xd, ldx, _opt(weight), wd,
                                          mean.data_ptr(), rstd.data_ptr(), M, N, dx.data_ptr(), lddx, _opt(dweight),
                                          _opt(dbias), _opt(workspace), 0 if workspace is None else workspace.numel(),
                                          _on(x, dev))
    if code:
        _raise(code, "fp8g_layer_norm_backward")


def layer_norm_backward(dy, x, weight, mean, rstd, weight_grads: bool = True):
    """-> (dx of x's type, dweight f32 [N], dbias f32 [N]); the last two are None without weight_grads."""
    dev, shape = x.device, x.shape
    dx = _empty(shape, dtype=x.dtype, device=dev)
    dw = db = None
    if weight_grads:
        dw = _empty(shape[-1], dtype=_F32, device=dev)
        db = _empty(shape[-1], dtype=_F32, device=dev)
    _norm_grad(dy, x, weight, mean, rstd, dx, shape[-1], dw, db, None)
    return dx, dw, db


# ------------------------------------------------------------------ gate

def _mask(mask, T: int) -> int:
    if mask.dtype not in (torch.bool, _U8) or mask.numel() != T or not mask.is_contiguous():
        _refuse(f"token_mask: bool or uint8 [{T}], contiguous")
    return mask.data_ptr()


def fp8g_moe_gate(logits, topk: int, topk_ids, topk_weights, counts, loss=None, renormalize: bool = True,
                  loss_coef: float = 0.01, token_mask=None, workspace=None) -> None:
    """logits [T,E] bf16 or f32 -> topk_ids int32 [T,topk], topk_weights f32 [T,topk], counts int32 [E], loss f32 [1]
    (or None).  token_mask: bool or uint8 [T], False for padding tokens.  workspace: a uint8 tensor of
    fp8g_moe_gate_workspace bytes (allocated if None)."""
    _need(logits.dim() == 2, "logits: [T,E]")
    T, E = logits.shape
    _vector(topk_ids, T * topk, _I32, "topk_ids")
    _vector(topk_weights, T * topk, _F32, "topk_weights")
    _vector(counts, E, _I32, "counts")
    if loss is not None:
        _vector(loss, 1, _F32, "loss")
    if workspace is not None:
        _scratch(workspace)
    _one_device(logits.get_device(), topk_ids, topk_weights, counts, loss, workspace)
    _gate(logits, topk, topk_ids, topk_weights, counts, loss, renormalize, loss_coef, token_mask, workspace)


def _gate(logits, topk, topk_ids, topk_weights, counts, loss, renormalize, loss_coef, token_mask, workspace) -> None:
    """The inputs' checks and the call."""
    code, ld = _dtype(logits, "logits"), _rows(logits, "logits")
    T, E = logits.shape
    mask = None if token_mask is None else _mask(token_mask, T)
    dev = logits.get_device()
    _one_device(dev, token_mask)
    if workspace is None:
        workspace = _workspace("fp8g_moe_gate_workspace", logits.device, T, E)
    st = lib().fp8g_moe_gate(logits.data_ptr(), code, T, E, ld, topk, 1 if renormalize else 0, mask, loss_coef,
                             topk_ids.data_ptr(), topk_weights.data_ptr(), counts.data_ptr(), _opt(loss),
                             _opt(workspace), 0 if workspace is None else workspace.numel(), _on(logits, dev))
    if st:
        _raise(st, "fp8g_moe_gate")


def moe_gate(logits, topk: int, renormalize: bool = True, loss_coef: float = 0.01, token_mask=None):
    """logits [T,E] -> (topk_ids int32 [T,topk], topk_weights f32 [T,topk], counts int32 [E], balance loss f32 [1])."""
    _need(logits.dim() == 2, "logits: [T,E]")
    T, E = logits.shape
    dev = logits.device
    ids = _empty((T, topk), dtype=_I32, device=dev)
    w = _empty((T, topk), dtype=_F32, device=dev)
    counts = _empty(E, dtype=_I32, device=dev)
    loss = _empty(1, dtype=_F32, device=dev)
    _gate(logits, topk, ids, w, counts, loss, renormalize, loss_coef, token_mask, None)
    return ids, w, counts, loss


def fp8g_moe_gate_backward(logits, topk_ids, counts, dweights, dloss, dlogits, renormalize: bool = True,
                           loss_coef: float = 0.01, token_mask=None) -> None:
    """dweights f32 [T,topk] and dloss f32 [1] (either may be None) -> dlogits [T,E] of logits' type."""
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
        _refuse("dlogits: logits' shape and type")
    ldd = _rows(dlogits, "dlogits")
    _one_device(logits.get_device(), dlogits)
    _gate_grad(logits, topk_ids, counts, dweights, dloss, dlogits, ldd, renormalize, loss_coef, token_mask)


def _gate_grad(logits, topk_ids, counts, dweights, dloss, dlogits, ldd, renormalize, loss_coef, token_mask) -> None:
    """The inputs' checks and the call."""
    code, ld = _dtype(logits, "logits"), _rows(logits, "logits")
    T, E = logits.shape
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        _refuse("topk_ids: int32 [T,topk]")
    topk = topk_ids.shape[1]
    _vector(topk_ids, T * topk, _I32, "topk_ids")
    _vector(counts, E, _I32, "counts")
    if dweights is not None:
        _vector(dweights, T * topk, _F32, "dweights")
    if dloss is not None:
        _vector(dloss, 1, _F32, "dloss")
    mask = None if token_mask is None else _mask(token_mask, T)
    dev = logits.get_device()
    _one_device(dev, topk_ids, counts, dweights, dloss, token_mask)
    st = lib().fp8g_moe_gate_backward(logits.data_ptr(), code, T, E, ld, topk, 1 if renormalize else 0, mask, loss_coef,
                                      topk_ids.data_ptr(), counts.data_ptr(), _opt(dweights), _opt(dloss),
                                      dlogits.data_ptr(), ldd, _on(logits, dev))
    if st:
        _raise(st, "fp8g_moe_gate_backward")


def moe_gate_backward(logits, topk_ids, counts, dweights=None, dloss=None, renormalize: bool = True,
                      loss_coef: float = 0.01, token_mask=None):
    """The gradient of moe_gate's weights and loss with respect to the logits -> dlogits [T,E]."""
    dlogits = _empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _gate_grad(logits, topk_ids, counts, dweights, dloss, dlogits, logits.shape[-1], renormalize, loss_coef, token_mask)
    return dlogits


# ------------------------------------------------------------------ combine

def fp8g_moe_combine(D, entry_row, weights, out, residual=None) -> None:
    """D bf16 [M,N], entry_row int32 [T,topk], weights f32 [T,topk] or None (1) -> out [T,N] bf16 or f32, plus
    residual [T,N] of out's type."""
    if out.dim() != 2 or out.shape[0] != entry_row.shape[0] or out.shape[1] != D.shape[-1]:
        _refuse("out: [T,N]")
    ldo = _rows(out, "out")
    _one_device(D.get_device(), out)
    _combine(D, entry_row, weights, out, ldo, residual)


def _combine(D, entry_row, weights, out, ldo: int, residual) -> None:
    """The inputs' checks and the call."""
    if D.dtype != torch.bfloat16:
        _refuse("D: bf16 [M,N]")
    code, ldd = _dtype(out, "out"), _rows(D, "D")
    M, N = D.shape
    if entry_row.dim() != 2:
        _refuse("entry_row: int32 [T,topk]")
    T, topk = entry_row.shape
    _vector(entry_row, T * topk, _I32, "entry_row")
    if weights is not None:
        _vector(weights, T * topk, _F32, "weights")
    ldr, res = 0, None
    if residual is not None:
        ldr, res = _rows(residual, "residual"), residual.data_ptr()
        if residual.shape != (T, N) or residual.dtype != out.dtype:
            _refuse("residual: out's shape and type")
    dev = D.get_device()
    _one_device(dev, entry_row, weights, residual)
    st = lib().fp8g_moe_combine(D.data_ptr(), M, N, ldd, entry_row.data_ptr(), T, topk, _opt(weights), res, ldr,
                                out.data_ptr(), code, ldo, _on(D, dev))
    if st:
        _raise(st, "fp8g_moe_combine")


def moe_combine(D, entry_row, weights=None, residual=None, out_dtype=None):
    """The experts' rows D back to their tokens -> out [T,N] of out_dtype (the residual's type, or bf16)."""
    dtype = out_dtype or (D.dtype if residual is None else residual.dtype)
    N = D.shape[-1]
    out = _empty((entry_row.shape[0], N), dtype=dtype, device=D.device)
    _combine(D, entry_row, weights, out, N, residual)
    return out


def fp8g_moe_combine_backward(dout, D, entry_row, row_token, weights, dD, dweights=None) -> None:
    """dout [T,N] bf16 or f32, D bf16 [M,N] (None if dweights is), entry_row int32 [T,topk], row_token int32 [M] ->
    dD bf16 [M,N] (padding rows zero), dweights f32 [T,topk] (or None)."""
    code, lddo, lddd = _dtype(dout, "dout"), _rows(dout, "dout"), _rows(dD, "dD")
    if dD.dtype != torch.bfloat16:
        _refuse("dD: bf16 [M,N]")
    M, N = dD.shape
    if entry_row.dim() != 2:
        _refuse("entry_row: int32 [T,topk]")
    T, topk = entry_row.shape
    if dout.shape != (T, N):
        _refuse("dout: [T,N]")
    if dweights is not None and D is None:
        _refuse("D: needed for dweights")
    ldd, d = 0, None
    if D is not None:
        ldd, d = _rows(D, "D"), D.data_ptr()
        if D.dtype != torch.bfloat16 or D.shape != dD.shape:
            _refuse("D: bf16 [M,N]")
    _vector(entry_row, T * topk, _I32, "entry_row")
    _vector(row_token, M, _I32, "row_token")
    if weights is not None:
        _vector(weights, T * topk, _F32, "weights")
    if dweights is not None:
        _vector(dweights, T * topk, _F32, "dweights")
    dev = dout.get_device()
    _one_device(dev, D, entry_row, row_token, weights, dD, dweights)
    st = lib().fp8g_moe_combine_backward(dout.data_ptr(), code, lddo, d, M, N, ldd, entry_row.data_ptr(),
                                         row_token.data_ptr(), T, topk, _opt(weights), dD.data_ptr(), lddd,
                                         _opt(dweights), _on(dout, dev))
    if st:
        _raise(st, "fp8g_moe_combine_backward")


def moe_combine_backward(dout, D, entry_row, row_token, weights=None):
    """-> (dD bf16 [M,N], dweights f32 [T,topk], or None without weights)."""
    dev = dout.device
    dD = _empty(D.shape, dtype=torch.bfloat16, device=dev)
    dw = None if weights is None else _empty(entry_row.shape, dtype=_F32, device=dev)
    fp8g_moe_combine_backward(dout, D, entry_row, row_token, weights, dD, dw)
    return dD, dw


# ------------------------------------------------------------------ gradient norm

class GradList:
    """The gradients of a program (and, for clipping out of place, the tensors that take the results), checked and
    listed once.  It holds the tensors and the memory they had, so nothing else comes to lie there.  A call refuses a
    list whose tensors have been given other memory since (``t.data = ...``, a ``resize_`` that grows): a program whose
    gradients move makes a new one.  (keep=False: for one call, before which nothing can move.)"""

    def __init__(self, grads, out=None, keep: bool = True):
        self.grads = grads = list(grads)
        self.out = grads if out is None else list(out)
        self.n = n = len(grads)
        _need(n > 0, "grads: at least one tensor")
        _need(len(self.out) == n, "out: a tensor for each gradient")
        self.device = grads[0].device
        self.device_index = dev = grads[0].get_device()
        self.codes = codes = []
        for t in grads:
            code = _DTYPES.get(t.dtype)
            if code is None or not t.is_contiguous():
                _refuse("grads: bf16 or f32, contiguous")
            if t.get_device() != dev or dev < 0:
                _refuse("grads: CUDA tensors on one device")
            codes.append(code)
        if out is not None:
            for t, o in zip(grads, self.out):
                if o.dtype != t.dtype or o.shape != t.shape or not o.is_contiguous():
                    _refuse("out: each gradient's shape and type, contiguous")
                if o.get_device() != dev:
                    _refuse("grads: CUDA tensors on one device")
        self.tensors = grads if out is None else grads + self.out
        self.places = [t.data_ptr() for t in self.tensors]
        self.sizes = [t.numel() for t in grads]
        if keep:
            self.memory = [t.untyped_storage() for t in self.tensors]
        self.indices = list(range(len(self.tensors))) if keep else None  # None: used at once, nothing moves
        self.disjoint = False  # whether the results are known to be (see check_results)
        self.ptrs = (ctypes.c_void_p * n)(*self.places[:n])
        self.out_ptrs = self.ptrs if out is None else (ctypes.c_void_p * n)(*self.places[n:])
        self.numels = (ctypes.c_int64 * n)(*self.sizes)
        self.dtypes = (ctypes.c_int32 * n)(*codes)
        b = ctypes.c_int64()
        _check(lib().fp8g_grad_norm_workspace(n, ctypes.byref(b)), "fp8g_grad_norm_workspace")
        self.workspace_bytes = b.value

    def __len__(self):
        return self.n

    def check_places(self) -> None:
        """Every tensor where it was when it was listed."""
        if self.indices is not None and not _all_at(self.tensors, self.places, self.indices):
            i = next(i for i, t in enumerate(self.tensors) if t.data_ptr() != self.places[i]) % self.n
            _refuse(f"grads: tensor {i} has moved since it was listed")

    def check_results(self) -> None:
        """No result overlaps another one, or a gradient that is not its own: it would be scaled twice, or read while it
        is written.  The places stay, so once is enough."""
        n, spans = self.n, []  # (start, end, written), empty tensors left out
        for at, to, size, code in zip(self.places, self.places[-n:], self.sizes, self.codes):
            if size:
                size <<= 1 + code
                spans.append((to, to + size, True))
                if at != to:
                    spans.append((at, at + size, False))
        spans.sort()
        written = known = 0  # the ends of the results, and of all tensors, so far
        for at, end, result in spans:
            if at < written or (result and at < known):
                _refuse("grads: a result overlaps another tensor of the list")
            if end > known:
                known = end
            if result:
                written = end
        self.disjoint = True


# Whether tensors[i].data_ptr() == places[i] for all indices i: on every call, so in one step where torch has it (300
# tensors 10 us, one by one 28).
_all_at = getattr(torch._C, "_tensors_data_ptrs_at_indices_equal",
                  lambda tensors, places, indices: [t.data_ptr() for t in tensors] == places)


def _norm_buffers(g: GradList, norm, workspace) -> None:
    _vector(norm, 1, _F32, "norm")
    if workspace is not None:
        _scratch(workspace)
    _one_device(g.device_index, norm, workspace)


def _workspace_of(g: GradList, workspace):
    return _empty(g.workspace_bytes, dtype=_U8, device=g.device) if workspace is None else workspace


def fp8g_grad_norm(grads: GradList, norm, workspace=None) -> None:
    """norm f32 [1] = the 2-norm of all gradients together."""
    _norm_buffers(grads, norm, workspace)
    _norm_of(grads, norm, workspace)


def _norm_of(g: GradList, norm, workspace) -> None:
    """The list's check and the call."""
    g.check_places()
    ws = _workspace_of(g, workspace)
    st = lib().fp8g_grad_norm(g.ptrs, g.numels, g.dtypes, g.n, norm.data_ptr(), ws.data_ptr(), ws.numel(),
                              _on(norm, g.device_index))
    if st:
        _raise(st, "fp8g_grad_norm")


def fp8g_clip_grad_norm(grads: GradList, max_norm: float, norm, eps: float = 1e-6, workspace=None) -> None:
    """norm f32 [1] as fp8g_grad_norm; every gradient times min(1, max_norm / (norm + eps)), into grads.out."""
    _norm_buffers(grads, norm, workspace)
    _clip(grads, max_norm, norm, eps, workspace)


def _clip(g: GradList, max_norm: float, norm, eps: float, workspace) -> None:
    """The list's checks and the call."""
    g.check_places()
    if not g.disjoint:
        g.check_results()
    ws = _workspace_of(g, workspace)
    st = lib().fp8g_clip_grad_norm(g.ptrs, g.out_ptrs, g.numels, g.dtypes, g.n, max_norm, eps, norm.data_ptr(),
                                   ws.data_ptr(), ws.numel(), _on(norm, g.device_index))
    if st:
        _raise(st, "fp8g_clip_grad_norm")


def _grad_list(grads) -> GradList:
    return grads if isinstance(grads, GradList) else GradList(grads, keep=False)


def grad_norm(grads) -> torch.Tensor:
    """grads: a GradList or a sequence of tensors -> their 2-norm, f32 [1] on the device."""
    g = _grad_list(grads)
    norm = _empty(1, dtype=_F32, device=g.device)
    _norm_of(g, norm, None)
    return norm


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + eps)), in place or, for a GradList with ``out``, into that
    -> the norm before clipping, f32 [1] on the device.  A plain sequence is checked and listed on every call: with 150
    tensors in place the call takes 141 us of the host, with a GradList 22 (1000 tensors: 830 and 74)."""
    g = _grad_list(grads)
    norm = _empty(1, dtype=_F32, device=g.device)
    _clip(g, max_norm, norm, eps, None)
    return norm
