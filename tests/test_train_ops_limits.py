"""Calls of the whole-block operators at the edge of what they take: refused by the host, before anything is launched."""

import ctypes

import pytest

from tests.test_train_ops_refusals import GLU_BWD, INVALID, NORM, NORM_BWD, ROUTE_BWD, _args, lib  # noqa: F401

P2 = 1 << 29


@pytest.mark.parametrize("N", [P2 + 1, (1 << 30) + 8, 0x7FFFFFF0])
def test_norm_columns_that_32_bits_do_not_count(lib, N):  # noqa: F811
    wide = {k: N for k in ("ldx", "ldf", "ldh", "ldy")}
    assert lib.fp8g_residual_rms_norm(*_args(NORM, dict(N=N, **wide))) == INVALID
    wide = {k: N for k in ("lddy", "lddh", "ldh", "ldf", "lddx", "lddf")}
    assert lib.fp8g_residual_rms_norm_backward(*_args(NORM_BWD, dict(N=N, wsb=1 << 50, **wide))) == INVALID
    n = ctypes.c_int64()
    assert lib.fp8g_residual_rms_norm_backward_workspace(4, N, ctypes.byref(n)) == INVALID


def test_norm_workspace_of_the_widest_rows(lib):  # noqa: F811
    n = ctypes.c_int64()
    assert lib.fp8g_residual_rms_norm_backward_workspace(1 << 20, P2, ctypes.byref(n)) == 0
    assert n.value >= 2 * P2 * 4 and n.value % (2 * P2 * 4) == 0


def test_results_in_place_of_an_input_keep_its_stride(lib):  # noqa: F811
    assert lib.fp8g_residual_rms_norm(*_args(NORM, dict(ldh=72))) == INVALID
    assert lib.fp8g_residual_rms_norm_backward(*_args(NORM_BWD, dict(lddx=72))) == INVALID
    assert lib.fp8g_swiglu_backward(*_args(GLU_BWD, dict(lddgu=264))) == INVALID
    assert lib.fp8g_moe_route_backward(*_args(ROUTE_BWD, dict(ldd=24))) == INVALID
