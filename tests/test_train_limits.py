"""The limits that moe_train.h names for the dense projection, at their last allowed and first
refused sizes (no GPU: an allowed size is refused for its workspace alone)."""

import ctypes
import os
import re

import pytest

from test_ext_abi import OK, UNSUPPORTED, WS_SMALL, at

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_train.h")

# (T, K, N) within the limits
INSIDE = [(1, (1 << 22) - 64, 64), (1, 64, (1 << 22) - 64), ((1 << 24) - 1, 64, 64), (1, 32768, 32704), (4095, 1 << 18, 64)]
# and one step outside: a width of 2^22, W, x or y of 2 GiB
OUTSIDE = [(1, 1 << 22, 64), (1, 64, 1 << 22), (1 << 24, 64, 64), (1, 32768, 32768), (4096, 1 << 18, 64), (4096, 64, 1 << 18)]


def calls(moe, T, K, N, dtype=1):
    from sparse_mixture_experts_route_amd import _lib
    lib = _lib.raw_lib()
    p = ctypes.byref(moe.Problem(T, K, 1, 1, N, dtype))
    a, small = [at(64 * i) for i in range(8)], ctypes.c_size_t(1)
    n = ctypes.c_size_t(0)
    sizes = [lib.moet_workspace_size(p, s, ctypes.byref(n)) for s in (moe.MOET_STAGE_LINEAR, moe.MOET_STAGE_LINEAR_BACKWARD)]
    return (lib.moet_linear(p, a[0], a[1], a[2], 1, a[3], a[4], a[5], a[6], small, None),
            lib.moet_linear_backward(p, a[0], a[1], a[2], 1, a[3], a[4], a[5], a[6], a[7], small, None), sizes)


@pytest.mark.parametrize("T,K,N", INSIDE)
def test_inside(moe, T, K, N):
    assert calls(moe, T, K, N) == (WS_SMALL, WS_SMALL, [OK, OK])


@pytest.mark.parametrize("T,K,N", OUTSIDE)
def test_outside(moe, T, K, N):
    assert calls(moe, T, K, N) == (UNSUPPORTED, UNSUPPORTED, [OK, OK])


def test_float32_has_sizes_and_no_calls(moe):
    assert calls(moe, 64, 128, 256, dtype=0) == (UNSUPPORTED, UNSUPPORTED, [OK, OK])


def test_the_header_names_the_limits():
    text = re.sub(r"\s*\n \* ", " ", open(HEADER).read())
    assert "reach 2 GiB, or K or N 2^22" in text and "moet_linear_backward has the same limits" in text
    assert "Any valid problem has a size" in text
