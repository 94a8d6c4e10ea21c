"""The router's general form with many picks: on both sides of the number up to which a row's contenders are looked for."""

import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_block_ops import _draw, _gen
from tests.test_gpu_train_ops import _check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [16, 17, 20, 24, 25, 28, 29, 32])
@pytest.mark.parametrize("E,groups,kept", [(640, 1, 1), (1024, 8, 3), (2048, 1, 1), (2016, 9, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_picks(k, E, groups, kept, score):
    need_gpu()
    T = 90
    kw = dict(score=score, groups=groups, topk_groups=kept)
    l, zero = _draw((T, E), "f32", 1), torch.zeros(E, device="cuda")
    few = _draw((T, E), "bf16", 2).mul_(2).round_().div_(2)  # many equal ones
    for logits in (l, few, l * 4 - 18):
        for bias in (None, zero, _draw((E,), "f32", 3, 0.05)):
            _check_route(logits, k, bias, **kw)
    l[torch.rand((T, E), generator=_gen(4), device="cuda") < 0.9] = -float("inf")
    l[3], l[4, 20:] = -float("inf"), -float("inf")
    for bias in (None, _draw((E,), "f32", 3, 0.05)):
        _check_route(l, k, bias, torch.arange(T, device="cuda") % 7 != 2, **kw)
