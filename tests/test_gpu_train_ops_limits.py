"""The whole-block operators where a call is allowed but unusual: offsets past 32 bits, more undecided rows than a CTA lists,
padded batches whose padding holds NaN, two calls at once on two streams, two graphs replayed at once, a gradient that two
parameters share."""

import itertools

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from oracle import train_ops as ot
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import _draw, _gen, _np
from tests.test_gpu_train_ops import _check_adam, _check_norm, _check_norm_grad, _check_route

pytestmark = pytest.mark.gpu

FAR = (1 << 27) + 8  # columns between two rows: 20 rows reach past 2^31 elements, 40 past 2^32


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def _far(rows, dtype, ld=FAR):
    return torch.empty((rows, ld), dtype=dtype, device="cuda")


@pytest.mark.parametrize("E,dtype", [(64, "bf16"), (256, "f32"), (800, "bf16")])
def test_route_rows_far_apart(E, dtype):
    l = _draw((40, E), dtype, 1)
    buf = _far(40, l.dtype)
    buf[:, :E] = l
    bias = _draw((E,), "f32", 2, 0.1)
    for score in ("sigmoid", "softmax"):
        ids, w, counts = _check_route(l, 4, bias, score=score)
        got = g.moe_route(buf[:, :E], 4, bias=bias, score=score)
        assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, counts)))
        dw = _draw((40, 4), "f32", 3)
        want = g.moe_route_backward(l, ids, dw, score=score)
        out = buf[:, 1024: 1024 + E]
        g.fp8g_moe_route_backward(buf[:, :E], ids, dw, out, score=score)
        assert torch.equal(out, want)
    check_status()


@pytest.mark.parametrize("N", [64, 4096, 7168, 12288, 17000])
def test_norm_rows_far_apart(N):
    M, P = 40, 1 << 15
    buf = _far(M, torch.bfloat16)
    x, f, h, y, dy, dh, dx, df = (buf[:, i * P: i * P + N] for i in range(8))
    for i, t in enumerate((x, f, dy, dh)):
        t.copy_(_draw((M, N), "bf16", i))
    w, gate, post = (_draw((N,), "f32", s, 0.3, 1.0) for s in (5, 6, 7))
    r, rf = (torch.empty(M, device="cuda") for _ in range(2))
    g.fp8g_residual_rms_norm(x, f, w, h, y, r, rf, gate=gate, post_norm=True, post_weight=post)
    sums = [torch.empty(N, device="cuda") for _ in range(3)]
    g.fp8g_residual_rms_norm_backward(dy, dh, h, f, r, rf, w, dx, df, *sums, gate=gate, post_norm=True, post_weight=post)
    check_status()
    x, f, dy, dh = (t.clone() for t in (x, f, dy, dh))
    want = g.residual_rms_norm(x, f, w, gate=gate, post_norm=True, post_weight=post)
    assert all(torch.equal(a, b) for a, b in zip((h, y, r, rf), want))
    want = g.residual_rms_norm_backward(dy, dh, h.clone(), f, r, rf, w, gate=gate, post_norm=True, post_weight=post)
    assert all(torch.equal(a, b) for a, b in zip((dx, df, *sums), want))


@pytest.mark.parametrize("N", [50, 4099])
def test_norm_rows_far_apart_and_off_the_grid(N):
    M, P = 40, 1 << 13
    buf = _far(M, torch.bfloat16, FAR + 3)
    x, f, h, y, dx, df = (buf[:, i * P: i * P + N] for i in range(6))
    x.copy_(_draw((M, N), "bf16", 1, 2.0))
    f.copy_(_draw((M, N), "bf16", 2))
    w = _draw((N,), "f32", 3, 0.3, 1.0)
    r = torch.empty(M, device="cuda")
    g.fp8g_residual_rms_norm(x, f, w, h, y, r)
    _check_norm(x, f, w, None, 1.0, False, None, (h, y, r, None), "bf16")
    dw = torch.empty(N, device="cuda")
    g.fp8g_residual_rms_norm_backward(y, x, h, f, r, None, w, dx, df, dw)
    check_status()
    _check_norm_grad(y, x, h, f, r, None, w, None, 1.0, False, None, (dx, df, dw, None, None), "bf16", "bf16")


def test_swiglu_rows_far_apart():
    M, F, P = 40, 384, 1 << 12
    buf = _far(M, torch.bfloat16)
    gu, h, dh, dgu = buf[:, : 2 * F], buf[:, P: P + F], buf[:, 2 * P: 2 * P + F], buf[:, 3 * P: 3 * P + 2 * F]
    gu.copy_(_draw((M, 2 * F), "bf16", 1, 2.0))
    dh.copy_(_draw((M, F), "bf16", 2))
    codes = _far(M, torch.uint8, FAR + 8)  # (rows of codes start on 16-byte boundaries)
    q, s = codes[:, :F], torch.empty((F // 128, M), device="cuda")
    g.fp8_swiglu_quantize_1x128(gu, q, s, h)
    g.fp8g_swiglu_backward(dh, gu, dgu)
    check_status()
    wq, ws, wh = g.swiglu_quantize_1x128(gu.clone(), keep=True)
    assert torch.equal(q, wq) and torch.equal(s, ws) and torch.equal(h, wh)
    assert torch.equal(dgu, g.swiglu_backward(dh.clone(), gu.clone())[0])


def test_swiglu_of_more_than_2_to_the_32_values():
    M, F = (1 << 21) + 33, 1024
    gu = torch.zeros((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    last = _draw((33, 2 * F), "bf16", 1, 2.0)
    gu[-33:] = last
    q, s, h = g.swiglu_quantize_1x128(gu, keep=True)
    wq, ws, wh = g.swiglu_quantize_1x128(last, keep=True)
    assert torch.equal(q[-33:], wq) and torch.equal(s[:, M - 33: M], ws[:, :33]) and torch.equal(h[-33:], wh)
    assert not q[:-33].any() and not h[:-33].any()


@pytest.mark.parametrize("bits,n", [(8, (1 << 32) + 517), (32, (1 << 31) + 517)])
def test_adamw_of_one_very_long_tensor(bits, n):
    """Values 2^32 apart draw the same dither, so the end of the long tensor is a short one's."""
    back = n - 517
    p, d = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    a, b = _draw((517,), "bf16", 1, 0.1), _draw((517,), "bf16", 2, 0.01)
    for at in (0, back):
        p[at: at + 517] = a
        d[at: at + 517] = b
    short = a.clone()
    one, long = g.AdamWList([short], [b], state_bits=bits), g.AdamWList([p], [d], state_bits=bits)
    for o in (one, long):
        g.adamw_step(o, 1e-2)
        g.adamw_step(o, 1e-2)
    check_status()
    for small, large in ((short, p), (one.m[0], long.m[0]), (one.v[0], long.v[0])):
        assert torch.equal(large[back:], small) and torch.equal(large[:512], small[:512])
        assert not large[640: 1 << 20].any() and not large[back - (1 << 20): back].any()


def _choices_in_doubt(scores, k, groups, kept):
    """The choices of a row that 64-bit scores allow.  Such a score is off by at most 8 2^-53 of itself (an exponential by 4
    roundings, a sum, a reciprocal and a product by one each), the sum of two by one more: group sums that lie within
    2 x 9 x 2^-53 of one another, relatively, have no order in 64 bits."""
    per = len(scores) // groups
    sums = np.sort(scores.reshape(groups, per), 1)[:, -2:].sum(1)
    border = np.sort(sums)[-kept]
    sure = np.flatnonzero(sums > border * (1 + 18 * 2.0 ** -53))
    doubt = np.flatnonzero(np.abs(sums / border - 1) <= 18 * 2.0 ** -53)
    for more in itertools.combinations(doubt, kept - len(sure)):
        e = np.concatenate([np.arange(i * per, i * per + per) for i in sorted([*sure, *more])])
        yield e[np.argsort(-scores[e], kind="stable")][:k]


@pytest.mark.parametrize("T,E,groups,kept", [(20000, 64, 8, 3), (11000, 256, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_where_every_row_is_close(T, E, groups, kept, score):
    """More rows than a CTA lists for its end have scores that fp32 does not tell apart.  (Some of 20000 rows have two groups
    whose sums, logits 0 + 4 and 2 + 2 steps off, differ by the score's curvature over those steps alone, some 10^-16: they may
    go either way.  What has no groups may not, for a step of a logit moves a score by more than 10^8 times its error.)"""
    base = torch.randn((T, 1), generator=_gen(5), device="cuda")
    near = base * (1 + torch.randint(0, 5, (T, E), generator=_gen(6), device="cuda") * 2.0 ** -23)
    bias = torch.zeros(E, device="cuda")
    ids, w, counts = g.moe_route(near, 4, bias=bias, score=score, groups=groups, topk_groups=kept)
    check_status()
    ids, s = ids.cpu().numpy(), ot.route_scores(_np(near), score)
    want, _, _ = ot.moe_route(_np(near), 4, _np(bias), score=score, groups=groups, topk_groups=kept)
    for t in np.flatnonzero((ids != want).any(1)):
        assert groups > 1 and any(np.array_equal(ids[t], c) for c in _choices_in_doubt(s[t], 4, groups, kept)), t
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.reshape(-1), minlength=E))
    assert np.allclose(_np(w), 0.25, rtol=1e-4, atol=0)  # (the chosen scores of a row are alike but for some 2^-20)


@pytest.mark.parametrize("E,groups,kept,k", [(640, 1, 1, 8), (1024, 8, 3, 8), (600, 6, 2, 16), (2016, 9, 4, 5), (513, 27, 5, 12),
                                             (576, 32, 7, 6), (2048, 1, 1, 17)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_many_experts_near_one_another(E, groups, kept, k, score):
    """More experts than lanes hold: fp32 says whose scores are needed in 64 bits, whatever the biases' size and sign."""
    T = 120
    kw = dict(score=score, groups=groups, topk_groups=kept)
    l, zero = torch.randn((T, E), generator=_gen(7), device="cuda"), torch.zeros(E, device="cuda")
    few = _draw((T, E), "bf16", 8).mul_(2).round_().div_(2)
    for logits in (few, l.bfloat16(), l * 4 + 18, l * 4 - 18, l):
        for bias in (None, zero, _draw((E,), "f32", 9, 1e-7), _draw((E,), "f32", 10, 3.0) + 100.0, -1e5 - _draw((E,), "f32", 11)):
            _check_route(logits, k, bias, **kw)
    level = torch.sigmoid(l[0]) if score == "sigmoid" else torch.softmax(l[0], 0)
    _check_route(l[:1].expand(T, E).contiguous(), k, 0.5 - level, **kw)  # every choice score is about 1/2
    base = torch.randn((T, 1), generator=_gen(5), device="cuda")
    near = base * (1 + torch.randint(0, 5, (T, E), generator=_gen(6), device="cuda") * 2.0 ** -23)
    if groups == 1:
        _check_route(near, k, zero, **kw)
    # ruled out: a logit, a bias, whole groups, all but a few
    l[torch.rand((T, E), generator=_gen(2), device="cuda") < 0.5] = -float("inf")
    l[3], l[4, 2:], l[5, : E // 2] = -float("inf"), -float("inf"), -float("inf")
    bias = _draw((E,), "f32", 3, 0.1)
    bias[:5], bias[E // 3: E // 2] = -float("inf"), -float("inf")
    for b in (None, bias):
        _check_route(l, k, b, torch.arange(T, device="cuda") % 7 != 2, **kw)
    l[7, 11], l[8, E - 1] = float("nan"), float("inf")
    ids, w, _ = g.moe_route(l, k, bias=bias, **kw)
    want, _, _ = ot.moe_route(_np(l), k, _np(bias), **kw)
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("T,E,k", [(12700, 64, 6), (13300, 64, 3), (5400, 128, 2), (5800, 96, 1)])
def test_route_where_shared_memory_is_just_below_48_kb(T, E, k):
    """The dynamic part alone is within what needs no leave, with the static part it is not."""
    _check_route(_draw((T, E), "f32", 1), k, _draw((E,), "f32", 2, 0.1))


@pytest.mark.parametrize("T,E,groups,kept", [(90, 64, 8, 4), (3000, 256, 8, 4), (40, 800, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_padding_of_nan(T, E, groups, kept, score):
    """What padding tokens hold reaches nothing: weights 0, no count, ids in range, no gradient."""
    l = _draw((T, E), "f32", 1)
    mask = torch.rand(T, generator=_gen(2), device="cuda") < 0.5
    mask[0], mask[-1] = True, False
    clean, bias = l.clone(), _draw((E,), "f32", 3, 0.1)
    l[~mask] = float("nan")
    kw = dict(score=score, groups=groups, topk_groups=kept)
    ids, w, counts = g.moe_route(l, 4, bias=bias, token_mask=mask, **kw)
    want = g.moe_route(clean, 4, bias=bias, token_mask=mask, **kw)
    assert torch.equal(ids[mask], want[0][mask]) and torch.equal(w, want[1]) and torch.equal(counts, want[2])
    assert not w[~mask].any() and int(ids.min()) >= 0 and int(ids.max()) < E
    dw = _draw((T, 4), "f32", 4)
    dw[~mask] = float("nan")
    got = g.moe_route_backward(l, ids, dw, score=score, token_mask=mask)
    assert torch.isfinite(got).all() and not got[~mask].any()
    assert torch.equal(got[mask], g.moe_route_backward(clean, want[0], dw, score=score, token_mask=mask)[mask])


def _calls(seed):
    """Each operator once, on tensors of its own; -> its results."""
    T, E, N, F = 3000, 64, 7168, 512
    l, bias = _draw((T, E), "bf16", seed), _draw((E,), "f32", seed + 1, 0.1)
    x, f, dy, dh = (_draw((300, N), "bf16", seed + i) for i in range(2, 6))
    w, dw = _draw((N,), "f32", seed + 6, 0.3, 1.0), _draw((T, 6), "f32", seed + 7)
    gu, da = _draw((500, 2 * F), "bf16", seed + 8), _draw((500, F), "bf16", seed + 9)
    first, d = _draw((70000,), "bf16", seed + 10, 0.1), _draw((70000,), "bf16", seed + 11, 0.01)
    p = first.clone()
    opt = g.AdamWList([p], [d], state_bits=8, masters=True)

    def call():
        ids, rw, counts = g.moe_route(l, 6, bias=bias, groups=8, topk_groups=4)
        h, y, r, rf = g.residual_rms_norm(x, f, w, gate=w, post_norm=True)
        out = [ids, rw, counts, g.moe_route_backward(l, ids, dw), h, y]
        out += [t for t in g.residual_rms_norm_backward(dy, dh, h, f, r, rf, w, w, 1.0, True) if t is not None]
        out += [*g.swiglu_quantize_1x128(gu, ld_sa=500, keep=True), *g.swiglu_backward(da, gu)]
        for t in (p, opt.masters[0], opt.m[0], opt.v[0], opt.m_scales[0], opt.v_scales[0], opt.step):
            t.zero_()  # (a run from the same state each time)
        p.copy_(first)
        opt.masters[0].copy_(first)
        g.adamw_step(opt, 1e-2)
        return out + [p, opt.masters[0], opt.m[0], opt.v[0], opt.step]

    return call


def test_two_calls_at_once_on_two_streams():
    calls = [_calls(10), _calls(50)]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i] = c()
    torch.cuda.synchronize()
    check_status()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_replayed_at_once():
    calls = [_calls(20), _calls(60)]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(c())
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    check_status()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_tensors_of_all_types_in_turn(bits):
    """A CTA's warps are at tensors of different types at the same time."""
    rng = np.random.default_rng(3)
    sizes = [int(n) for n in rng.integers(0, 60000, 60)]
    kinds = [(("bf16", "f32")[a], ("bf16", "f32")[b]) for a, b in rng.integers(0, 2, (60, 2))]
    params = [_draw((n,), k[0], i, 0.1) for i, (n, k) in enumerate(zip(sizes, kinds))]
    grads = [_draw((n,), k[1], 100 + i, 0.01) for i, (n, k) in enumerate(zip(sizes, kinds))]
    before = [p.clone() for p in params]
    masters = [p.float() if p.dtype == torch.bfloat16 and i % 3 == 0 else None for i, p in enumerate(params)]
    first = [None if t is None else t.clone() for t in masters]
    opt = g.AdamWList(params, grads, masters=masters, state_bits=bits)
    g.adamw_step(opt, 1e-2)
    check_status()
    for i in range(60):
        z, zs = torch.zeros_like(opt.m[i]), None if bits == 32 else torch.zeros_like(opt.m_scales[i])
        _check_adam((before[i], first[i], z, z, zs, zs),
                    (params[i], masters[i], opt.m[i], opt.v[i], opt.m_scales[i], opt.v_scales[i]), grads[i], 1, 1e-2, 0.9,
                    0.999, 1e-8, float(np.float32(0.01)), 1.0, bits, f"tensor {i}")


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_gradient_that_two_parameters_share(bits):
    d = _draw((3001,), "bf16", 1, 0.01)
    params = [_draw((3001,), "f32", 2, 0.1), _draw((3001,), "bf16", 3, 0.1)]
    before = [p.clone() for p in params]
    opt = g.AdamWList(params, [d, d], state_bits=bits, weight_decay=[0.0, 0.5])
    g.adamw_step(opt, 1e-2)
    z = torch.zeros_like(opt.m[0])
    zs = None if bits == 32 else torch.zeros_like(opt.m_scales[0])
    for i, decay in enumerate((0.0, 0.5)):
        _check_adam((before[i], None, z, z, zs, zs), (params[i], None, opt.m[i], opt.v[i], opt.m_scales[i], opt.v_scales[i]),
                    d, 1, 1e-2, 0.9, 0.999, 1e-8, decay, 1.0, bits, f"parameter {i}")


def test_adamw_of_empty_tensors_alone():
    """The step is counted."""
    e = torch.empty(0, device="cuda")
    opt = g.AdamWList([e], [e.clone()])
    g.adamw_step(opt, 1e-2)
    check_status()
    assert int(opt.step) == 1


def test_oracle_is_the_one_that_was_checked():
    """(The route's ids of equal logits are ascending, which every comparison above leans on.)"""
    ids, _, _ = ot.moe_route(np.zeros((2, 8)), 3)
    assert ids.tolist() == [[0, 1, 2]] * 2
    assert _np(g.moe_route(torch.zeros((2, 8), device="cuda"), 3)[0]).tolist() == [[0, 1, 2]] * 2
