"""Clipping of more than 256 MB of gradients (the 64 KB chunks) with tables of every size, mixed types, tensors that start
anywhere, in place and apart, against sums and products in 64 bits.

The norm's bound is that of test_gpu_block_ops.py: a thread adds n / (256 * 608) squares one after another, and forty
roundings cover the groups' and the partial sums' joins and the root; a result has twice that and its type's rounding.
"""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from tests.gpu_util import check_status, need_gpu
from tests.test_gpu_block_ops import DT, U

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    need_gpu()


def _views(sizes, kinds, gaps, values, seed):
    """Views of those sizes in a flat buffer for each type, `gaps` values of NaN before each; random where `values`."""
    room = {k: sum(n + p for n, kk, p in zip(sizes, kinds, gaps) if kk == k) + 16 for k in set(kinds)}
    flat = {k: torch.full((n,), float("nan"), dtype=DT[k], device="cuda") for k, n in sorted(room.items())}
    at, out = {k: 0 for k in flat}, []
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for n, k, p in zip(sizes, kinds, gaps):
        t = flat[k][at[k] + p: at[k] + p + n]
        if values:
            t.copy_(torch.randn(n, generator=gen, device="cuda") * 0.01 + 1e-4)
        at[k] += p + n
        out.append(t)
    return out, flat


@pytest.mark.parametrize("count", [100, 500, 1100])
@pytest.mark.parametrize("kinds", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("place", ["in place", "apart, as far off the grid", "apart, otherwise off the grid"])
def test_clip_above_256_mb(count, kinds, place):
    rng = np.random.default_rng(count)
    share = np.exp(rng.normal(0.0, 2.0, count))
    sizes = [int(n) for n in np.maximum(1, share / share.sum() * (150e6 if kinds == "bf16" else 80e6))]
    sizes[3], sizes[7] = 1, 40961  # a single value; a little more than a chunk of either type
    kinds = [kinds if kinds != "mixed" else ("bf16", "f32")[int(i)] for i in rng.integers(0, 2, count)]
    if len(set(kinds)) > 1:  # above the limit with any draw of the types
        sizes = [2 * n if k == "bf16" else n for n, k in zip(sizes, kinds)]
    assert sum(n * (4 if k == "f32" else 2) for n, k in zip(sizes, kinds)) > 256 << 20
    gaps = [int(p) for p in rng.integers(0, 9, count)]
    grads, flat = _views(sizes, kinds, gaps, True, count)
    want = [t.double() for t in grads]
    rnorm = float(torch.stack([t.square().sum() for t in want]).sum().sqrt())
    max_norm = 0.3 * rnorm
    coef = min(1.0, max_norm / (rnorm + 1e-6))
    if place == "in place":
        lst, buffers = g.GradList(grads), flat
    else:
        other = gaps if place == "apart, as far off the grid" else [(p * 5 + 3) % 9 for p in gaps]
        out, buffers = _views(sizes, kinds, other, False, 0)
        lst = g.GradList(grads, out)
    k = (sum(sizes) / (256 * 608) + 40) * U
    norm = g.grad_norm(lst)
    assert abs(float(norm) - rnorm) <= k * rnorm
    assert torch.equal(g.clip_grad_norm(lst, max_norm), norm)
    for t, r, kind in zip(lst.out, want, kinds):
        r = r * coef
        tol = (2 * k + (2.0 ** -8 if kind == "bf16" else 0.0)) * r.abs() + 1e-37
        assert bool(((t.double() - r).abs() <= tol).all())
    for kind, buf in buffers.items():  # nothing else was written
        assert int(torch.isnan(buf).sum()) == buf.numel() - sum(n for n, kk in zip(sizes, kinds) if kk == kind)
    check_status()
