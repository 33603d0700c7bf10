"""Sizes past a limit of the operators are refused on the host, before anything is
enqueued (no call here launches a kernel: the addresses are never dereferenced)."""

import ctypes

import pytest

from test_ext_abi import UNSUPPORTED, WS_SMALL, P, at, f32


@pytest.fixture(scope="module")
def lib(moe):
    from sparse_mixture_experts_route_amd import _lib
    return _lib.raw_lib()


def backward_status(lib, moe, balanced, **size):
    """Status of the backward pass with a workspace of one byte."""
    x, wr, W1, W2, dy, mk, dx, dwr, db, dW1, dW2, ls, ct, mp, ws = (at(16 * i) for i in range(15))
    one = ctypes.c_size_t(1)
    if balanced:
        return lib.moex_backward_balanced(P(moe, **size), x, wr, W1, W2, dy, mk, f32(0.01), dx, dwr, db, dW1, dW2, ls,
                                          ct, mp, ws, one, None)
    return lib.moe_backward(P(moe, **size), x, wr, W1, W2, dy, dx, dwr, db, dW1, dW2, None, mp, ws, one, None)


PAST = [  # the first size that a product of the backward cannot address, and one below it
    (dict(T=65536, k=8, d=2048, de=256, E=64), dict(T=65535, k=8, d=2048, de=256, E=64)),      # rows of d_model
    (dict(T=65536, k=8, d=64, de=2048, E=8), dict(T=65535, k=8, d=64, de=2048, E=8)),          # rows of d_expert
    (dict(T=64, k=1, d=32768, de=32768, E=8), dict(T=64, k=1, d=32768, de=32704, E=8)),        # an expert's weight
    (dict(T=1 << 22, k=1, d=64, de=64, E=200), dict(T=(1 << 22) - 1, k=1, d=64, de=64, E=200)),  # logits' gradient
    (dict(T=64, k=1, d=1 << 22, de=64, E=256), dict(T=64, k=1, d=(1 << 22) - 64, de=64, E=256)),  # w_router
]


@pytest.mark.parametrize("balanced", [False, True], ids=["moe_backward", "moex_backward_balanced"])
@pytest.mark.parametrize("past,below", PAST, ids=["d_model", "d_expert", "weight", "logits", "router"])
def test_backward_refuses_what_its_products_cannot_address(moe, lib, past, below, balanced):
    assert backward_status(lib, moe, balanced, **below) == WS_SMALL
    assert backward_status(lib, moe, balanced, **past) == UNSUPPORTED


def test_experts_refuse_what_their_launches_cannot_hold(moe, lib):
    """Before the first product, or the first weight, is enqueued."""
    a = [at(i << 16) for i in range(11)]  # 1 PiB apart
    one = ctypes.c_size_t(1)
    wide = dict(T=(1 << 24) - 1, k=128, E=128, d=128, de=1 << 21)  # 2^52 hidden values
    for size, want in ((wide, UNSUPPORTED), (dict(wide, T=1 << 13), WS_SMALL)):
        assert lib.moex_grouped_ffn_fp8(P(moe, **size), *a[:10], one, None) == want
        assert lib.moex_forward_fp8(P(moe, **size), *a, one, None) == want
    n = 1 << 19  # 2^38 values of an expert
    assert lib.moex_quantize_experts(P(moe, E=1, k=1, d=n, de=n), *a[:6], None) == UNSUPPORTED
