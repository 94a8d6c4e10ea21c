"""The router gives a row the same bits wherever it is decided: rows in doubt go to a CTA's end or, where there are more of
them than it lists, to the warp that has met them, and which ones do is a matter of timing.  A softmax's sum in 64 bits has
to be formed in the same order in both."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_block_gb300 as g
from tests.gpu_util import check_status, need_gpu

pytestmark = pytest.mark.gpu


def _rows_on_a_border(rows, E, seed):
    """Logits whose softmax has 1 / sum in the middle between two floats but for some roundings of 64 bits, so that another
    order of the sum's terms can round it to the other one; and a second choice in doubt."""
    rng = np.random.default_rng(seed)
    l = rng.uniform(-8.0, -1.0, (rows, E)).astype(np.float32)
    l[:, 0], l[:, 1], l[:, 2] = 0.0, -0.5, -0.5 * (1 + 2.0 ** -23)
    l[:, -2:] = -np.inf
    total = np.exp(l.astype(np.longdouble)).sum(1)
    below = np.nextafter((1 / total).astype(np.float32), np.float32(0))
    middle = (below.astype(np.longdouble) + np.nextafter(below, np.float32(0))) / 2
    for at in (-2, -1):  # two small terms fill the sum up to 1 / middle
        rest = 1 / middle - total
        term = np.log(rest).astype(np.float32)
        l[:, at] = np.where(np.exp(term.astype(np.longdouble)) > rest, np.nextafter(term, np.float32(-np.inf)), term)
        total = total + np.exp(l[:, at].astype(np.longdouble))
    return l


@pytest.mark.parametrize("E", [64, 160, 256])
def test_rows_in_doubt_beyond_a_ctas_list(E):
    need_gpu()
    distinct, times = 500, 60
    l = torch.from_numpy(np.tile(_rows_on_a_border(distinct, E, 1), (times, 1))).cuda()
    ids, w, _ = g.moe_route(l, 2, bias=torch.zeros(E, device="cuda"), score="softmax", renormalize=False)
    check_status()
    ids, w = ids.view(times, distinct, 2), w.view(times, distinct, 2)
    assert torch.equal(ids, ids[:1].expand_as(ids)) and torch.equal(w, w[:1].expand_as(w))
