"""The shapes that the routing of moe_permute_capacity may have are those that the calls it serves accept (host checks, no GPU)."""
import ctypes

import pytest

import bit_mixed_precision_router_b200 as moe
from bit_mixed_precision_router_b200 import ExpertsT, RoutingT

INVALID, SHAPE, WS = 1, 2, 3
A = 0x10000  # a fake, 16-byte aligned device address


@pytest.fixture(scope="module")
def lib():
    from bit_mixed_precision_router_b200 import build
    build.build()
    return moe.load()


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_grouped_ffn_with_more_choices_than_experts(lib, fmt):
    r, ex = RoutingT(A, A, A, A, A, A), ExpertsT(fmt, A, A, A, A, A, A)
    call = lambda T, E, k: lib.moe_grouped_ffn(A, ctypes.byref(r), ctypes.byref(ex), A, T, 256, 128, E, k, A, None, 0, None)
    assert call(4, 8, 2) == WS    # accepted up to the workspace, which is missing
    assert call(4, 2, 8) == WS    # a rank with two experts
    assert call(4, 1, 32) == WS
    assert call(4, 2, 33) == SHAPE
    assert call(4, 2, 0) == SHAPE
    assert call(4, 0, 2) == SHAPE
    assert call(4, 1025, 2) == SHAPE
    assert call(-1, 2, 8) == INVALID
    assert call((1 << 31) // 8, 2, 8) == SHAPE


def test_combine_with_more_choices_than_experts(lib):
    r = RoutingT(A, A, A, A, A, A)
    assert lib.moe_combine(A, ctypes.byref(r), None, 0, 256, 32, A, None) == 0
