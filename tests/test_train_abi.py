"""What trains the layer's surroundings, on the host: include/moe_train.h is exported,
workspaces are sized, and bad arguments are refused before anything reaches the GPU
(no call here launches a kernel)."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

from test_ext_abi import BAD, INVALID, OK, UNSUPPORTED, WS_SMALL, P, at

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_train.h")
BIG = 1 << 40


def declared():
    return sorted(set(re.findall(r"^moe_status_t\s+(moet_\w+)\s*\(", open(HEADER).read(), re.M)))


def test_header_and_library_agree(libmoe_path):
    out = subprocess.run(["nm", "-D", "--defined-only", libmoe_path], capture_output=True, text=True).stdout
    assert sorted(set(re.findall(r"\bT (moet_\w+)", out))) == declared()
    assert len(declared()) == 11


@pytest.fixture(scope="module")
def lib(moe):
    from sparse_mixture_experts_route_amd import _lib
    return _lib.raw_lib()


def size_of(moe, stage, T=64, d=128, E=8, k=2, de=256, dtype=1):
    return moe.moet_workspace_size(moe.Problem(T, d, E, k, de, dtype), stage)


def refuses_each_missing(call, args, needed, *tail):
    for i in needed:
        a = list(args)
        a[i] = None
        assert call(*a, *tail) == INVALID, i


def test_workspace_sizes(moe, lib):
    n = ctypes.c_size_t(0)
    for stage in range(3):
        assert lib.moet_workspace_size(P(moe), stage, ctypes.byref(n)) == OK and n.value > 0
        for b in BAD:
            assert lib.moet_workspace_size(P(moe, **b), stage, ctypes.byref(n)) != OK
    for stage in (-1, 3):
        assert lib.moet_workspace_size(P(moe), stage, ctypes.byref(n)) == INVALID
    assert lib.moet_workspace_size(P(moe), 0, None) == INVALID
    assert lib.moet_workspace_size(None, 0, ctypes.byref(n)) == INVALID
    # dU and its column sums
    assert size_of(moe, 2, T=4096, d=2048, de=8192) >= 4096 * 8192 * 2


def test_dispatch_refuses(moe, lib):
    need = size_of(moe, 0)
    a = [at(i) for i in range(9)]  # topk_idx, weight, x, counts, offsets, perm, inv, x_perm, ws
    f = lambda *v, **k: lib.moet_dispatch(P(moe, **k), *v)  # noqa: E731
    assert f(*a, need - 1, None) == WS_SMALL
    refuses_each_missing(f, a, (0, 2, 3, 4, 5, 6, 7, 8), need, None)
    for i, j in ((7, 2), (6, 5), (4, 3), (8, 0), (3, 1)):
        b = list(a)
        b[i] = b[j]
        assert f(*b, need, None) == INVALID, (i, j)
    b = list(a)
    b[2] += 8
    assert f(*b, need, None) == INVALID
    for bad in BAD:
        assert f(*a, BIG, None, **bad) != OK


def test_dispatch_backward_and_combine_refuse(moe, lib):
    a = [at(i) for i in range(7)]  # dx_perm, inv, x, weight, residual, dx, dweight
    f = lambda *v, **k: lib.moet_dispatch_backward(P(moe, **k), *v, None)  # noqa: E731
    refuses_each_missing(f, a, (0, 1, 2, 5, 6))
    for i, j in ((5, 0), (5, 4), (6, 3), (6, 5)):
        b = list(a)
        b[i] = b[j]
        assert f(*b) == INVALID, (i, j)
    c = [at(i) for i in range(5)]  # y_perm, inv, gate, residual, y
    g = lambda *v, **k: lib.moet_combine(P(moe, **k), *v, None)  # noqa: E731
    refuses_each_missing(g, c, (0, 1, 4))
    for j in (0, 2, 3):
        b = list(c)
        b[4] = b[j]
        assert g(*b) == INVALID
    for bad in BAD:
        assert f(*a, **bad) != OK and g(*c, **bad) != OK


def test_combine_backward_and_gate_backward_refuse(moe, lib):
    a = [at(i) for i in range(6)]  # dy, inv, y_perm, gate, dy_perm, dgate
    f = lambda *v, **k: lib.moet_combine_backward(P(moe, **k), *v, None)  # noqa: E731
    refuses_each_missing(f, a, (0, 1, 2, 4, 5))
    for i, j in ((4, 0), (4, 2), (5, 3), (5, 4)):
        b = list(a)
        b[i] = b[j]
        assert f(*b) == INVALID, (i, j)
    c = [at(i) for i in range(5)]  # logits, topk_idx, dgate, add, dlogits
    g = lambda *v, **k: lib.moet_gate_backward(P(moe, **k), *v, None)  # noqa: E731
    refuses_each_missing(g, c, (0, 1, 2, 4))
    for j in (0, 2, 3):
        b = list(c)
        b[4] = b[j]
        assert g(*b) == INVALID
    for bad in BAD:
        assert f(*a, **bad) != OK and g(*c, **bad) != OK


def test_linear_refuses(moe, lib):
    need = size_of(moe, 1)
    x, W, b, r, u, y, ws = (at(i) for i in range(7))
    f = lambda *v, **k: lib.moet_linear(P(moe, **k), *v)  # noqa: E731
    ok = [x, W, b, 1, r, u, y, ws]
    assert f(*ok, need - 1, None) == WS_SMALL
    refuses_each_missing(f, ok, (0, 1, 6, 7), need, None)
    for act in (-1, 4):
        assert f(x, W, b, act, r, u, y, ws, need, None) == INVALID
    for i, j in ((6, 4), (6, 0), (5, 6), (7, 1)):
        a = list(ok)
        a[i] = a[j]
        assert f(*a, need, None) == INVALID, (i, j)
    assert f(*ok, BIG, None, dtype=0) == UNSUPPORTED
    far = [at(64 * i) if isinstance(v, int) and v > 3 else v for i, v in enumerate(ok)]
    for big in (dict(T=1 << 20, d=1024), dict(T=1 << 20, de=1024, d=64), dict(d=32768, de=32768), dict(T=1, d=1 << 22),
                dict(T=1, d=64, de=1 << 22)):
        assert f(*far, BIG, None, **big) == UNSUPPORTED, big
    assert f(*far, 1, None, T=(1 << 20) - 1, d=1024, de=64) == WS_SMALL


def test_linear_backward_refuses(moe, lib):
    need = size_of(moe, 2)
    x, W, u, dy, dx, dW, db, ws = (at(i) for i in range(8))
    f = lambda *v, **k: lib.moet_linear_backward(P(moe, **k), *v)  # noqa: E731
    ok = [x, W, u, 1, dy, dx, dW, db, ws]
    assert f(*ok, need - 1, None) == WS_SMALL
    refuses_each_missing(f, ok, (0, 1, 2, 4, 8), need, None)
    assert f(x, W, u, 1, dy, None, None, None, ws, need, None) == INVALID
    assert f(x, W, None, 2, dy, dx, dW, db, ws, need, None) == INVALID  # an activation's slope needs u
    for i, j in ((5, 0), (5, 4), (6, 1), (7, 5), (8, 2)):
        a = list(ok)
        a[i] = a[j]
        assert f(*a, need, None) == INVALID, (i, j)
    assert f(*ok, BIG, None, dtype=0) == UNSUPPORTED


def entry(moe, i=0, n=100, bf16=True, small=False, **kw):
    """A list entry with addresses of its own (never dereferenced)."""
    b = 16 * i
    e = moe.Tensor(param=at(b), grad=at(b + 1), master=at(b + 2) if bf16 else None, m=at(b + 3), v=at(b + 4),
                   m_scale=at(b + 5) if small else None, v_scale=at(b + 6) if small else None, n=n,
                   param_dtype=1 if bf16 else 0, grad_dtype=1, lr_factor=1.0, weight_decay=0.1)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def arr(moe, *e):
    return (moe.Tensor * max(1, len(e)))(*e)


def adamw_status(moe, lib, entries, counter=at(1000), lr_scale=None, grad_scale=None, **kw):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, seed=1)
    o.update(kw)
    return lib.moet_adamw(arr(moe, *entries), len(entries), ctypes.byref(moe.AdamWOptions(**o)), counter, lr_scale,
                          grad_scale, None)


def test_adamw_refuses(moe, lib):
    one = entry(moe)
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
                dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-16), dict(eps=float("inf"))):
        assert adamw_status(moe, lib, [one], **bad) == INVALID, bad
    assert adamw_status(moe, lib, [one], counter=None) == INVALID
    assert adamw_status(moe, lib, [one], counter=at(1000) + 4) == INVALID
    assert lib.moet_adamw(None, 1, ctypes.byref(moe.AdamWOptions(1e-3, 0.9, 0.99, 1e-8, 0)), at(9), None, None, None) == INVALID
    assert lib.moet_adamw(arr(moe, one), 1, None, at(1000), None, None, None) == INVALID
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(master=None), dict(n=-1),
               dict(param_dtype=2), dict(grad_dtype=-1), dict(lr_factor=float("nan")), dict(lr_factor=-1.0),
               dict(weight_decay=-0.1), dict(weight_decay=float("inf")), dict(param=at(0) + 2), dict(m_scale=at(5)),
               dict(param_dtype=0)):
        assert adamw_status(moe, lib, [entry(moe, **kw)]) == INVALID, kw
    assert adamw_status(moe, lib, [entry(moe, n=1 << 41)]) == UNSUPPORTED
    assert adamw_status(moe, lib, [entry(moe, i, n=1 << 40) for i in range(2)]) == UNSUPPORTED
    assert adamw_status(moe, lib, [entry(moe, i) for i in range(1025)]) == INVALID
    # overlaps: within a tensor, between tensors, with the counter and the factors
    for kw in (dict(grad=at(0)), dict(v=at(3)), dict(master=at(0) + 100), dict(m=at(1000))):
        assert adamw_status(moe, lib, [entry(moe, **kw)]) == INVALID, kw
    assert adamw_status(moe, lib, [entry(moe), entry(moe, 1, param=at(0) + 192)]) == INVALID
    assert adamw_status(moe, lib, [entry(moe, small=True, v_scale=at(5))]) == INVALID
    assert adamw_status(moe, lib, [one], lr_scale=at(0)) == INVALID
    assert adamw_status(moe, lib, [one], grad_scale=at(1000)) == INVALID


def test_clipped_step_refuses(moe, lib):
    one, ws, ok = arr(moe, entry(moe)), at(300), moe.MOET_GRAD_NORM_WS_BYTES
    o = ctypes.byref(moe.AdamWOptions(1e-3, 0.9, 0.99, 1e-8, 1))
    f = lambda *a: lib.moet_adamw_clipped(*a, None)  # noqa: E731
    d = ctypes.c_double
    for bad in (0.0, -1.0, float("nan")):
        assert f(one, 1, o, at(1000), None, d(bad), at(301), at(302), ws, ok) == INVALID
    for a in ((None, 1, o, at(1000), None, d(1), at(301), at(302), ws, ok), (one, 1, None, at(1000), None, d(1), at(301), None, ws, ok),
              (one, 1, o, None, None, d(1), at(301), None, ws, ok), (one, 1, o, at(1000), None, d(1), None, None, ws, ok),
              (one, 1, o, at(1000), None, d(1), at(301), None, None, ok), (one, 1, o, at(1000), None, d(1), at(301), at(301), ws, ok),
              (one, 1, o, at(1000), None, d(1), at(1000), None, ws, ok), (one, 1, o, at(1000), at(301), d(1), at(301), None, ws, ok),
              (one, 1, o, at(1000), None, d(1), at(1), None, ws, ok), (one, 1, o, at(1000), None, d(1), at(301), None, at(3), ok)):
        assert f(*a) == INVALID
    assert f(one, 1, o, at(1000), None, d(1), at(301), None, ws, ok - 1) == WS_SMALL


def test_grad_norm_refuses(moe, lib):
    one = arr(moe, entry(moe))
    f = lib.moet_grad_norm
    ws, ok = at(300), moe.MOET_GRAD_NORM_WS_BYTES
    d = ctypes.c_double
    for bad in (0.0, -1.0, float("nan")):
        assert f(one, 1, d(bad), at(301), at(302), ws, ok, None) == INVALID
    assert f(one, 1, d(1.0), None, at(302), ws, ok, None) == INVALID
    assert f(one, 1, d(1.0), at(301), at(302), None, ok, None) == INVALID
    assert f(one, 1, d(1.0), at(301), at(302), ws, ok - 1, None) == WS_SMALL
    assert f(one, 1, d(1.0), at(301), at(301), ws, ok, None) == INVALID
    assert f(one, 1, d(1.0), at(1), at(302), ws, ok, None) == INVALID  # norm over the gradient
    assert f(one, -1, d(1.0), at(301), at(302), ws, ok, None) == INVALID
    assert f(None, 1, d(1.0), at(301), at(302), ws, ok, None) == INVALID


def test_binding_checks_tensors(moe):
    p = moe.make_problem(4, 64, 2, 1, 64, torch.float32)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        moe.moet_combine(p, x, x, None, None, x)
    with pytest.raises(ValueError, match="required"):
        moe.moet_linear(p, None, x, None, 0, None, None, x, x)
    with pytest.raises(ValueError, match="GPU"):
        moe.AdamW([x])
    with pytest.raises(ValueError, match="expected 1 to"):
        moe.AdamW([])
    with pytest.raises(ValueError, match="params lack"):
        moe.MoETrainBlock(4, 64, 8, 1, 64, {"gain": x})
    with pytest.raises(ValueError, match="dense expert has"):
        moe.MoETrainBlock(4, 64, 8, 1, 64, {"gain": x, "V1": x})
    with pytest.raises(moe.MoEError):
        moe.moet_workspace_size(p, 17)
