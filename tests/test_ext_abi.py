"""The operators around the layer on the host: include/moe_ext.h is exported,
workspaces are sized, and bad arguments are refused before anything reaches the
GPU (no call here launches a kernel)."""

import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_ext.h")
OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
GB = 1 << 30


def declared():
    return sorted(set(re.findall(r"^moe_status_t\s+(moex_\w+)\s*\(", open(HEADER).read(), re.M)))


def test_header_and_library_agree(libmoe_path):
    out = subprocess.run(["nm", "-D", "--defined-only", libmoe_path], capture_output=True, text=True).stdout
    assert sorted(set(re.findall(r"\bT (moex_\w+)", out))) == declared()
    assert len(declared()) == 9


@pytest.fixture(scope="module")
def lib(moe):
    from sparse_mixture_experts_route_amd import _lib
    return _lib.raw_lib()


def P(moe, T=64, d=128, E=8, k=2, de=256, dtype=1):
    return ctypes.byref(moe.Problem(T, d, E, k, de, dtype))


def at(i, off=0):
    """A fake 16-byte aligned device address, 16 GiB apart from the others (never dereferenced)."""
    return (i + 1) * 16 * GB + off


def f32(v):
    return ctypes.c_float(v)


BAD = [dict(T=0), dict(d=96), dict(E=257, k=2), dict(k=9), dict(dtype=5)]


def test_workspace_sizes(moe, lib):
    n = ctypes.c_size_t(0)
    for stage in range(5):
        assert lib.moex_workspace_size(P(moe), stage, ctypes.byref(n)) == OK and n.value > 0
        for b in BAD:
            assert lib.moex_workspace_size(P(moe, **b), stage, ctypes.byref(n)) != OK
    assert lib.moex_workspace_size(P(moe), 5, ctypes.byref(n)) == INVALID
    assert lib.moex_workspace_size(P(moe), -1, ctypes.byref(n)) == INVALID
    assert lib.moex_workspace_size(P(moe), 0, None) == INVALID
    assert lib.moex_workspace_size(None, 0, ctypes.byref(n)) == INVALID
    p = moe.make_problem(4096, 2048, 8, 2, 8192, "bf16")
    R = 8192
    assert moe.moex_workspace_size(p, moe.MOEX_STAGE_FFN_FP8) >= R * (8192 + 64)
    assert moe.moex_workspace_size(p, moe.MOEX_STAGE_TRAIN_BALANCED) > moe.moe_workspace_size(p, moe.MOE_STAGE_TRAIN)


def test_norm_refuses(moe, lib):
    f = lambda *a, **k: lib.moex_add_rmsnorm(P(moe, **k), *a)  # noqa: E731
    x, r, g, h, y, y8, ys, rs = (at(i) for i in range(8))
    e = f32(1e-6)
    assert f(None, r, g, e, h, y, y8, ys, rs, None) == INVALID
    assert f(x, r, None, e, h, y, y8, ys, rs, None) == INVALID
    assert f(x, r, g, e, None, y, y8, ys, rs, None) == INVALID       # residual without h
    assert f(x, None, g, e, h, y, y8, ys, rs, None) == INVALID       # h without residual
    assert f(x, r, g, e, h, y, y8, None, rs, None) == INVALID        # codes without scales
    assert f(x, None, g, e, None, None, None, None, None, None) == INVALID  # no output
    for bad in (-1e-6, float("nan"), float("inf")):
        assert f(x, r, g, f32(bad), h, y, y8, ys, rs, None) == INVALID
    assert f(x + 8, r, g, e, h, y, y8, ys, rs, None) == INVALID      # misaligned
    assert f(x, r, g, e, x, y, y8, ys, rs, None) == INVALID          # h overlaps x
    assert f(x, r, g, e, h, r + 64 * 128 * 2 - 16, y8, ys, rs, None) == INVALID  # y's start overlaps residual's end
    assert f(x, r, g, e, h, y, y + 16, ys, rs, None) == INVALID      # two outputs overlap
    assert f(x, r, g, e, h, y, y8, ys, rs, None, d=32768 + 64) == UNSUPPORTED
    for b in BAD:
        assert f(x, r, g, e, h, y, y8, ys, rs, None, **b) != OK


def test_norm_backward_refuses(moe, lib):
    f = lambda *a, **k: lib.moex_add_rmsnorm_backward(P(moe, **k), *a)  # noqa: E731
    h, g, rs, dy, dh, dx, dg, ws = (at(i) for i in range(8))
    need = moe.moex_workspace_size(moe.Problem(64, 128, 8, 2, 256, 1), moe.MOEX_STAGE_NORM_BACKWARD)
    assert f(h, g, rs, dy, dh, dx, dg, ws, need - 1, None) == WS_SMALL
    for i in (0, 1, 2, 3, 5, 6, 7):
        a = [h, g, rs, dy, dh, dx, dg, ws]
        a[i] = None
        assert f(*a, need, None) == INVALID, i
    assert f(h, g, rs, dy, dh, dy, dg, ws, need, None) == INVALID    # dx overlaps dy
    assert f(h, g, rs, dy, dh, dx, dg, h, need, None) == INVALID     # ws overlaps h
    assert f(h, g, rs, dy, dh, dx, dg + 4, ws, need, None) == INVALID
    assert f(h, g, rs, dy, dh, dx, dg, ws, 1 << 40, None, d=65536) == UNSUPPORTED


def test_quantize_refuses(moe, lib):
    x, x8, xs = at(0), at(1), at(2)
    assert lib.moex_quantize_rows(P(moe), None, x8, xs, None) == INVALID
    assert lib.moex_quantize_rows(P(moe), x, None, xs, None) == INVALID
    assert lib.moex_quantize_rows(P(moe), x, x8, None, None) == INVALID
    assert lib.moex_quantize_rows(P(moe), x, x, xs, None) == INVALID
    a = [at(i) for i in range(6)]
    assert lib.moex_quantize_experts(P(moe, dtype=0), *a, None) == UNSUPPORTED
    for i in range(6):
        b = list(a)
        b[i] = None
        assert lib.moex_quantize_experts(P(moe), *b, None) == INVALID
    b = list(a)
    b[2] = a[0]
    assert lib.moex_quantize_experts(P(moe), *b, None) == INVALID


def test_balance_refuses(moe, lib):
    f = lambda *a, **k: lib.moex_balance_loss(P(moe, **k), *a)  # noqa: E731
    lg, ix, mk, ls, ct, mp, dl, ws = (at(i) for i in range(8))
    need = moe.moex_workspace_size(moe.Problem(64, 128, 8, 2, 256, 1), moe.MOEX_STAGE_BALANCE)
    c = f32(0.01)
    assert f(lg, ix, mk, c, ls, ct, mp, dl, ws, need - 1, None) == WS_SMALL
    for i in (0, 1, 3, 4, 5, 7):
        a = [lg, ix, mk, ls, ct, mp, dl, ws]
        a[i] = None
        assert f(*a[:3], c, *a[3:], need, None) == INVALID, i
    for bad in (float("nan"), float("inf")):
        assert f(lg, ix, mk, f32(bad), ls, ct, mp, dl, ws, need, None) == INVALID
    assert f(lg, ix, mk, c, ls, ct, mp, lg, ws, need, None) == INVALID  # dlogits over logits
    assert f(lg, ix, mk, c, ls, ct, ct, dl, ws, need, None) == INVALID
    for b in BAD:
        assert f(lg, ix, mk, c, ls, ct, mp, dl, ws, need, None, **b) != OK


def test_backward_balanced_refuses(moe, lib):
    f = lambda *a, **k: lib.moex_backward_balanced(P(moe, **k), *a)  # noqa: E731
    n = [at(i) for i in range(16)]
    x, wr, W1, W2, dy, mk, dx, dwr, db, dW1, dW2, ls, ct, mp, ws = n[:15]
    c = f32(0.01)
    need = moe.moex_workspace_size(moe.Problem(64, 128, 8, 2, 256, 1), moe.MOEX_STAGE_TRAIN_BALANCED)
    args = [x, wr, W1, W2, dy, mk, c, dx, dwr, db, dW1, dW2, ls, ct, mp, ws]
    assert f(*args, need - 1, None) == WS_SMALL
    for i in (0, 1, 2, 3, 4, 7, 8, 10, 11, 12, 15):
        a = list(args)
        a[i] = None
        assert f(*a, need, None) == INVALID, i
    assert f(*args, need, None, dtype=0) == UNSUPPORTED
    assert f(*args, 1 << 40, None, E=12) == UNSUPPORTED
    assert f(*args, 1 << 40, None, E=16, k=9) == UNSUPPORTED
    a = list(args)
    a[7] = dy
    assert f(*a, need, None) == INVALID


def test_ffn_and_forward_refuse(moe, lib):
    a = [at(i) for i in range(10)]  # x8, x_scale, perm, offsets, W1q, W1s, W2q, W2s, y_perm, ws
    need = moe.moex_workspace_size(moe.Problem(64, 128, 8, 2, 256, 1), moe.MOEX_STAGE_FFN_FP8)
    assert lib.moex_grouped_ffn_fp8(P(moe), *a, need - 1, None) == WS_SMALL
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9):
        b = list(a)
        b[i] = None
        assert lib.moex_grouped_ffn_fp8(P(moe), *b, need, None) == INVALID, i
    b = list(a)
    b[8] = a[0]
    assert lib.moex_grouped_ffn_fp8(P(moe), *b, need, None) == INVALID
    assert lib.moex_grouped_ffn_fp8(P(moe, dtype=0), *a, need, None) == UNSUPPORTED
    # codes of 2 GiB: rows without and with the permutation, and one expert's weight
    assert lib.moex_grouped_ffn_fp8(P(moe, T=1 << 20, d=2048, k=1), *a, 1 << 44, None) == UNSUPPORTED
    b = list(a)
    b[2] = None
    assert lib.moex_grouped_ffn_fp8(P(moe, T=1 << 19, d=2048, k=2), *b, 1 << 44, None) == UNSUPPORTED
    assert lib.moex_grouped_ffn_fp8(P(moe, d=32768, de=65536, E=1, k=1), *a, 1 << 44, None) == UNSUPPORTED
    a = [at(i) for i in range(11)]  # x, x8, x_scale, w_router, bias, W1q, W1s, W2q, W2s, y, ws
    need = moe.moex_workspace_size(moe.Problem(64, 128, 8, 2, 256, 1), moe.MOEX_STAGE_FORWARD_FP8)
    assert lib.moex_forward_fp8(P(moe), *a, need - 1, None) == WS_SMALL
    for i in (0, 3, 5, 6, 7, 8, 9, 10):
        b = list(a)
        b[i] = None
        assert lib.moex_forward_fp8(P(moe), *b, need, None) == INVALID, i
    b = list(a)
    b[2] = None  # codes without scales
    assert lib.moex_forward_fp8(P(moe), *b, need, None) == INVALID
    assert lib.moex_forward_fp8(P(moe, dtype=0), *a, need, None) == UNSUPPORTED


def test_binding_checks_tensors(moe):
    import torch
    p = moe.make_problem(4, 64, 1, 1, 64, torch.float32)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        moe.moex_quantize_rows(p, x, x, x)
    with pytest.raises(ValueError, match="required"):
        moe.moex_add_rmsnorm(p, None, None, x, 1e-6, None, x, None, None, None)
    with pytest.raises(TypeError):
        moe.moex_add_rmsnorm(p, 3, None, x, 1e-6, None, x, None, None, None)
    with pytest.raises(moe.MoEError):
        moe.moex_workspace_size(p, 17)
    assert moe.code_pitch(320) == 384 and moe.scale_pitch(320) == 16 and moe.scale_pitch(2112) == 32


def test_coef_whose_product_with_E_overflows_is_refused(moe, lib):
    """coef E multiplies the zeros of masked rows: infinity there would be NaN."""
    n = ctypes.c_size_t(1 << 40)
    a = [at(i) for i in range(16)]
    for c in (1e38, -1e38):
        assert lib.moex_balance_loss(P(moe), a[0], a[1], a[2], f32(c), *a[3:8], n, None) == INVALID
        assert lib.moex_backward_balanced(P(moe), *a[:6], f32(c), *a[6:15], n, None) == INVALID


def test_workspace_of_another_form_is_refused(moe, lib, monkeypatch):
    """The form of the products is read at every call: a workspace sized for one that needs less is too small."""
    n = ctypes.c_size_t(0)
    big = dict(T=4096, d=2048, E=8, k=2, de=8192)
    monkeypatch.setenv("MOE_FP8_TILES", "0")
    for stage in (2, 3):
        assert lib.moex_workspace_size(P(moe, **big), stage, ctypes.byref(n)) == OK
        size = n.value
        monkeypatch.setenv("MOE_FP8_TILES", "1")
        a = [at(i) for i in range(11)]
        assert lib.moex_workspace_size(P(moe, **big), stage, ctypes.byref(n)) == OK and n.value > size
        have = ctypes.c_size_t(size)
        if stage == 2:
            assert lib.moex_grouped_ffn_fp8(P(moe, **big), *a[:10], have, None) == WS_SMALL
        else:
            assert lib.moex_forward_fp8(P(moe, **big), *a, have, None) == WS_SMALL
        monkeypatch.setenv("MOE_FP8_TILES", "0")
