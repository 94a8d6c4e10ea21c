"""The training operators' argument checks, in the library (before anything is launched) and in the binding; and the
calls that have nothing to do.  No GPU needed."""

import ctypes

import pytest
import torch

import moe_grouped_gemm_block_gb300 as g

INVALID, ALIGN = 1, 2
P = 1 << 20  # an aligned fake device address, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return g.lib()


def _args(defaults, kw):
    assert set(kw) <= set(defaults)
    return tuple({**defaults, **kw}.values())


NORM = dict(x=P, xd=0, M=4, N=64, ldx=64, w=P, b=P, wd=1, eps=1e-5, y=P, yd=0, ldy=64, mean=P, rstd=P, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(xd=2), INVALID), (dict(yd=-1), INVALID), (dict(wd=7), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=63), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(M=1 << 31), INVALID),
    (dict(x=P + 1), ALIGN), (dict(w=P + 2), ALIGN), (dict(mean=P + 2), ALIGN), (dict(y=P + 2, yd=1), ALIGN),
    (dict(M=0, x=None, y=None), 0),
])
def test_layer_norm(lib, kw, want):
    assert lib.fp8g_layer_norm(*_args(NORM, kw)) == want


NORM_BWD = dict(dy=P, yd=0, lddy=64, x=P, xd=0, ldx=64, w=P, wd=1, mean=P, rstd=P, M=4, N=64, dx=P, lddx=64, dw=P,
                db=P, ws=P, wsb=BIG, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(yd=3), INVALID), (dict(lddy=8), INVALID), (dict(lddx=8), INVALID), (dict(mean=None), INVALID),
    (dict(dx=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=16), INVALID), (dict(M=-1), INVALID),
    (dict(ws=P + 8), ALIGN), (dict(dw=P + 1), ALIGN), (dict(dx=P + 1), ALIGN),
    (dict(M=0, dy=None, x=None, mean=None, rstd=None, dx=None, dw=None, db=None, ws=None), 0),
])
def test_layer_norm_backward(lib, kw, want):
    assert lib.fp8g_layer_norm_backward(*_args(NORM_BWD, kw)) == want


GATE = dict(l=P, d=1, T=50000, E=8, ldl=8, k=2, renorm=1, mask=None, coef=0.01, ids=P, w=P, counts=P, loss=P, ws=P,
            wsb=BIG, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=2), INVALID), (dict(E=0), INVALID), (dict(E=2049, ldl=2049), INVALID), (dict(ldl=7), INVALID),
    (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(E=64, ldl=64, k=33), INVALID), (dict(renorm=2), INVALID),
    (dict(T=-1), INVALID), (dict(T=(1 << 31) - 1, k=8), INVALID), (dict(counts=None), INVALID),
    (dict(ids=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=8), INVALID),
    (dict(ids=P + 2), ALIGN), (dict(l=P + 2), ALIGN), (dict(ws=P + 4), ALIGN),
])
def test_gate(lib, kw, want):
    assert lib.fp8g_moe_gate(*_args(GATE, kw)) == want


GATE_BWD = dict(l=P, d=1, T=4, E=8, ldl=8, k=2, renorm=1, mask=None, coef=0.01, ids=P, counts=P, dw=P, dloss=P, dl=P,
                ldd=8, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=2), INVALID), (dict(ldd=7), INVALID), (dict(k=9), INVALID), (dict(ids=None), INVALID),
    (dict(dl=None), INVALID), (dict(dl=P + 2), ALIGN), (dict(dw=P + 1), ALIGN), (dict(T=0, l=None, dl=None), 0),
])
def test_gate_backward(lib, kw, want):
    assert lib.fp8g_moe_gate_backward(*_args(GATE_BWD, kw)) == want


COMBINE = dict(D=P, M=128, N=64, ldd=64, rows=P, T=4, k=2, w=P, res=None, ldr=0, out=P, od=0, ldo=64, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=60, ldd=64, ldo=64), INVALID), (dict(ldd=56), INVALID), (dict(ldo=56), INVALID), (dict(k=0), INVALID),
    (dict(od=5), INVALID), (dict(D=None), INVALID), (dict(rows=None), INVALID), (dict(res=P, ldr=32), INVALID),
    (dict(M=-1), INVALID), (dict(T=1 << 30, k=4), INVALID),
    (dict(D=P + 8), ALIGN), (dict(out=P + 2), ALIGN), (dict(ldd=68), ALIGN), (dict(res=P + 4, ldr=64), ALIGN),
    (dict(T=0, D=None, out=None, rows=None), 0),
])
def test_combine(lib, kw, want):
    assert lib.fp8g_moe_combine(*_args(COMBINE, kw)) == want


COMBINE_BWD = dict(dout=P, dd=0, lddo=64, D=P, M=128, N=64, ldd=64, rows=P, tokens=P, T=4, k=2, w=P, dD=P, lddd=64,
                   dw=P, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=60), INVALID), (dict(lddd=56), INVALID), (dict(lddo=56), INVALID), (dict(tokens=None), INVALID),
    (dict(D=None), INVALID), (dict(dD=None), INVALID), (dict(dout=None), INVALID), (dict(dd=2), INVALID),
    (dict(dD=P + 8), ALIGN), (dict(lddo=68), ALIGN), (dict(dw=P + 2), ALIGN),
    (dict(M=0, T=0, dout=None, D=None, dD=None, rows=None, tokens=None), 0),
])
def test_combine_backward(lib, kw, want):
    assert lib.fp8g_moe_combine_backward(*_args(COMBINE_BWD, kw)) == want


def _clip(lib, ptrs=(P, P), numels=(8, 8), dtypes=(1, 0), outs=(P, P), max_norm=1.0, eps=1e-6, norm=P, ws=P, wsb=BIG):
    n = len(numels)
    return lib.fp8g_clip_grad_norm((ctypes.c_void_p * n)(*ptrs), (ctypes.c_void_p * n)(*outs),
                                   (ctypes.c_int64 * n)(*numels), (ctypes.c_int32 * n)(*dtypes), n, max_norm, eps, norm,
                                   ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(numels=(8, -1)), INVALID), (dict(dtypes=(1, 2)), INVALID), (dict(ptrs=(P, None)), INVALID),
    (dict(outs=(None, P)), INVALID), (dict(max_norm=-1.0), INVALID), (dict(max_norm=float("nan")), INVALID),
    (dict(eps=-1.0), INVALID), (dict(norm=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=64), INVALID),
    (dict(numels=(1 << 42, 1)), INVALID),
    (dict(ptrs=(P + 2, P)), ALIGN), (dict(outs=(P, P + 1)), ALIGN), (dict(ws=P + 4), ALIGN), (dict(norm=P + 1), ALIGN),
])
def test_clip(lib, kw, want):
    assert _clip(lib, **kw) == want


def test_null_tables(lib):
    assert lib.fp8g_grad_norm(None, None, None, 2, P, P, BIG, None) == INVALID
    assert lib.fp8g_grad_norm(None, None, None, -1, P, P, BIG, None) == INVALID
    assert lib.fp8g_grad_norm_workspace(4, None) == INVALID
    assert lib.fp8g_moe_gate_workspace(4, 0, ctypes.byref(ctypes.c_int64())) == INVALID
    n = ctypes.c_int64(-1)
    assert lib.fp8g_moe_gate_workspace(4, 8, ctypes.byref(n)) == 0 and n.value == 0  # few tokens: none needed
    assert lib.fp8g_moe_gate_workspace(50000, 8, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.fp8g_layer_norm_backward_workspace(4, 0, ctypes.byref(ctypes.c_int64())) == INVALID


def test_valid_arguments_without_a_gpu_report_an_error(lib):
    if torch.cuda.is_available():
        pytest.skip("GPU present: covered by the GPU tests")
    for name, args in (("fp8g_layer_norm", NORM), ("fp8g_layer_norm_backward", NORM_BWD), ("fp8g_moe_gate", GATE),
                       ("fp8g_moe_gate_backward", GATE_BWD), ("fp8g_moe_combine", COMBINE),
                       ("fp8g_moe_combine_backward", COMBINE_BWD)):
        assert getattr(lib, name)(*args.values()) in (3, 4), name
    assert _clip(lib) in (3, 4)


# ---- the binding: ValueError before the library is called

def _f32(*shape):
    return torch.zeros(shape)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_layer_norm():
    with pytest.raises(ValueError, match="x: bf16 or f32"):
        g.layer_norm(torch.zeros(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="weight"):
        g.layer_norm(_f32(4, 8), _f32(7))
    with pytest.raises(ValueError, match="one type"):
        g.layer_norm(_f32(4, 8), _f32(8), _bf16(8))
    with pytest.raises(ValueError, match="rows contiguous"):
        g.layer_norm(_f32(8, 4).t())
    with pytest.raises(ValueError, match="CUDA tensors"):
        g.layer_norm(_f32(4, 8), _f32(8), _f32(8))
    with pytest.raises(ValueError, match="mean"):
        g.layer_norm_backward(_f32(4, 8), _f32(4, 8), _f32(8), _f32(3), _f32(4))
    with pytest.raises(ValueError, match="x's shape"):
        g.layer_norm_backward(_f32(4, 7), _f32(4, 8), _f32(8), _f32(4), _f32(4))


def test_binding_gate():
    with pytest.raises(ValueError, match="logits"):
        g.moe_gate(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="token_mask"):
        g.moe_gate(_f32(4, 8), 2, token_mask=torch.ones(3, dtype=torch.bool))
    with pytest.raises(ValueError, match="topk_ids"):
        g.fp8g_moe_gate(_f32(4, 8), 2, _i32(4, 3), _f32(4, 2), _i32(8))
    with pytest.raises(ValueError, match="CUDA tensors"):
        g.moe_gate(_f32(4, 8), 2)
    with pytest.raises(ValueError, match="counts"):
        g.moe_gate_backward(_f32(4, 8), _i32(4, 2), _i32(7), _f32(4, 2))
    with pytest.raises(ValueError, match="dweights"):
        g.moe_gate_backward(_f32(4, 8), _i32(4, 2), _i32(8), _f32(4, 3))


def test_binding_combine():
    with pytest.raises(ValueError, match="D: bf16"):
        g.moe_combine(_f32(128, 64), _i32(4, 2), _f32(4, 2), out_dtype=torch.float32)
    with pytest.raises(ValueError, match="weights"):
        g.moe_combine(_bf16(128, 64), _i32(4, 2), _f32(4, 3))
    with pytest.raises(ValueError, match="residual"):
        g.moe_combine(_bf16(128, 64), _i32(4, 2), _f32(4, 2), residual=_f32(4, 32))
    with pytest.raises(ValueError, match="row_token"):
        g.moe_combine_backward(_bf16(4, 64), _bf16(128, 64), _i32(4, 2), _i32(64), _f32(4, 2))
    with pytest.raises(ValueError, match="CUDA tensors"):
        g.moe_combine(_bf16(128, 64), _i32(4, 2), _f32(4, 2))


def test_binding_clip():
    with pytest.raises(ValueError, match="at least one"):
        g.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        g.clip_grad_norm([_f32(4, 8).t()], 1.0)
    with pytest.raises(ValueError, match="bf16 or f32"):
        g.grad_norm([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="CUDA tensors"):
        g.clip_grad_norm([_f32(8)], 1.0)
    with pytest.raises(ValueError, match="a tensor for each"):
        g.GradList([_f32(8)], [])


# ---- tensors of a GPU that is not the current one: the library launches on the current one

class _Elsewhere(torch.Tensor):
    """A host tensor that says it lies on GPU 1."""

    def get_device(self):
        return 1


def _there(t):
    return t.as_subclass(_Elsewhere)


class _NeverCalled:
    """Stands for the library: its size queries answer, a launch fails the test."""

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 0
        return lambda *a: pytest.fail(f"{name} was launched")


def _calls_elsewhere():
    x, v, m, ids = _there(_f32(4, 8)), _there(_f32(8)), _there(_f32(4)), _there(_i32(4, 2))
    D, w, tok = _there(_bf16(128, 8)), _there(_f32(4, 2)), _there(_i32(128))
    return {
        "fp8g_layer_norm": lambda: g.fp8g_layer_norm(x, v, v, x, m, m),
        "layer_norm": lambda: g.layer_norm(x, v, v),
        "fp8g_layer_norm_backward": lambda: g.fp8g_layer_norm_backward(x, x, v, m, m, x, v, v),
        "layer_norm_backward": lambda: g.layer_norm_backward(x, x, v, m, m),
        "fp8g_moe_gate": lambda: g.fp8g_moe_gate(x, 2, ids, w, _there(_i32(8))),
        "moe_gate": lambda: g.moe_gate(x, 2),
        "fp8g_moe_gate_backward": lambda: g.fp8g_moe_gate_backward(x, ids, _there(_i32(8)), w, None, x),
        "moe_gate_backward": lambda: g.moe_gate_backward(x, ids, _there(_i32(8)), w),
        "fp8g_moe_combine": lambda: g.fp8g_moe_combine(D, ids, w, x),
        "moe_combine": lambda: g.moe_combine(D, ids, w),
        "fp8g_moe_combine_backward": lambda: g.fp8g_moe_combine_backward(x, D, ids, tok, w, D, w),
        "fp8g_grad_norm": lambda: g.fp8g_grad_norm(g.GradList([x]), _there(_f32(1)),
                                                   _there(torch.zeros(8, dtype=torch.uint8))),
        "fp8g_clip_grad_norm": lambda: g.fp8g_clip_grad_norm(g.GradList([x]), 1.0, _there(_f32(1)), 1e-6,
                                                             _there(torch.zeros(8, dtype=torch.uint8))),
        "quantize_1x128": lambda: g._stream(x),  # what every GEMM and quantiser call takes its stream from
    }


@pytest.mark.parametrize("name", list(_calls_elsewhere()))
def test_tensors_of_another_gpu_than_the_current_one(name, monkeypatch):
    from moe_grouped_gemm_block_gb300 import block_ops as bo
    monkeypatch.setattr(g, "_current_device", lambda: 0)
    monkeypatch.setattr(bo, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type("S", (), {"cuda_stream": 0}))
    monkeypatch.setattr(bo, "lib", _NeverCalled)
    monkeypatch.setattr(bo, "_workspace_bytes", lambda *a: 0)
    with pytest.raises(ValueError, match="current device"):
        _calls_elsewhere()[name]()


# ---- gradients whose storage has been replaced since they were listed

class _Here(torch.Tensor):
    """A host tensor that says it lies on GPU 0."""

    def get_device(self):
        return 0


def _move_data(t):
    t.data = t.data.clone()


def _grow(t):
    t.resize_(1 << 20)


@pytest.mark.parametrize("move", [_move_data, _grow])
@pytest.mark.parametrize("which", ["gradient", "result"])
@pytest.mark.parametrize("call", ["norm", "clip"])
def test_a_listed_gradient_that_has_moved(move, which, call, monkeypatch):
    from moe_grouped_gemm_block_gb300 import block_ops as bo
    monkeypatch.setattr(g, "_current_device", lambda: 0)
    monkeypatch.setattr(bo, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(bo, "lib", _NeverCalled)
    grads = [_f32(8).as_subclass(_Here), _bf16(5, 3).as_subclass(_Here)]
    out = [t.clone() for t in grads]
    lst = g.GradList(grads, out)
    move(grads[1] if which == "gradient" or call == "norm" else out[1])
    one = [_f32(1).as_subclass(_Here), torch.zeros(8, dtype=torch.uint8).as_subclass(_Here)]
    with pytest.raises(ValueError, match="tensor 1 has moved"):
        g.fp8g_grad_norm(lst, *one) if call == "norm" else g.fp8g_clip_grad_norm(lst, 1.0, one[0], 1e-6, one[1])


def test_a_list_keeps_the_memory_that_it_names():
    t = torch.zeros(64, 4).as_subclass(_Here)
    lst, address = g.GradList([t]), t.data_ptr()
    t.data = torch.zeros(64, 4)
    assert [m.data_ptr() for m in lst.memory] == [address] != [t.data_ptr()]  # no later tensor can lie there


# ---- results that overlap another tensor of the list: scaled twice, or read while they are written

def _overlap_lists():
    a, b = _f32(64), _f32(64)
    return {
        "the same gradient twice, in place": ([a, a], None, True),
        "views that share values, in place": ([a[:40], a[39:]], None, True),
        "neighbouring views, in place": ([a[:40], a[40:]], None, False),
        "a gradient twice, results apart": ([a, a], [b[:64], _f32(64)], False),
        "one result for two gradients": ([a[:32], a[32:]], [b[:32], b[:32]], True),
        "a result over another gradient": ([a[:32], a[32:]], [b[:32], a[:32]], True),
        "a result over a part of its own gradient": ([a[:32]], [a[4:36]], True),
        "in place beside apart": ([a[:32], a[32:]], [a[:32], b[:32]], False),
        "an empty tensor anywhere": ([a, a[5:5]], None, False),
    }


@pytest.mark.parametrize("name", list(_overlap_lists()))
def test_overlapping_results(name, monkeypatch):
    from moe_grouped_gemm_block_gb300 import block_ops as bo
    grads, out, refused = _overlap_lists()[name]
    launched = []

    class Lib:
        def __getattr__(self, fn):
            return lambda *a: launched.append(fn) or 0

    monkeypatch.setattr(g, "_current_device", lambda: 0)
    monkeypatch.setattr(bo, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(bo, "lib", Lib)
    here = lambda ts: None if ts is None else [t.as_subclass(_Here) for t in ts]
    lst = g.GradList(here(grads), here(out))
    one = [_f32(1).as_subclass(_Here), torch.zeros(8, dtype=torch.uint8).as_subclass(_Here)]
    g.fp8g_grad_norm(lst, *one)  # the norm alone writes to none of them
    assert launched[-1] == "fp8g_grad_norm"
    if refused:
        with pytest.raises(ValueError, match="overlaps"):
            g.fp8g_clip_grad_norm(lst, 1.0, one[0], 1e-6, one[1])
    else:
        g.fp8g_clip_grad_norm(lst, 1.0, one[0], 1e-6, one[1])
        g.fp8g_clip_grad_norm(lst, 1.0, one[0], 1e-6, one[1])
    assert ("fp8g_clip_grad_norm" in launched) is not refused
