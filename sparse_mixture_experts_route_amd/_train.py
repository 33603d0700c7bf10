"""What trains the layer's surroundings (include/moe_train.h): argument marshalling.

The functions carry the C names and argument order and check each tensor's
type, size and device, as the operators around the layer do. The list calls
take an array of `Tensor` entries, which `tensor_entry` makes.
"""

from __future__ import annotations

import ctypes

import torch

from . import _ext, _lib
from ._ext import _BF16, _F32, _I32, _call, _device, _opt, _ptr, _rows, _ws
from ._lib import MOE_DTYPE_BF16, MOE_DTYPE_F32, Problem

MOET_STAGE_DISPATCH = 0
MOET_STAGE_LINEAR = 1
MOET_STAGE_LINEAR_BACKWARD = 2

MOET_ACT_NONE = 0
MOET_ACT_GELU = 1
MOET_ACT_SILU = 2
MOET_ACT_RELU = 3

MOET_MAX_TENSORS = 1024
MOET_GRAD_NORM_WS_BYTES = 8704

_c = _lib.raw_lib()


class Tensor(ctypes.Structure):
    """An entry of a list: moet_tensor_t."""

    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "master", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("lr_factor", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class AdamWOptions(ctypes.Structure):
    """moet_adamw_t."""

    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("seed", ctypes.c_uint32)]


def _declare():
    P, A, O = ctypes.POINTER(Problem), ctypes.POINTER(Tensor), ctypes.POINTER(AdamWOptions)
    vp, i32, sz, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_double
    sigs = {
        "moet_workspace_size": [P, i32, ctypes.POINTER(sz)],
        "moet_dispatch": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moet_dispatch_backward": [P, vp, vp, vp, vp, vp, vp, vp, vp],
        "moet_combine": [P, vp, vp, vp, vp, vp, vp],
        "moet_combine_backward": [P, vp, vp, vp, vp, vp, vp, vp],
        "moet_gate_backward": [P, vp, vp, vp, vp, vp, vp],
        "moet_linear": [P, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp],
        "moet_linear_backward": [P, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp],
        "moet_adamw": [A, i32, O, vp, vp, vp, vp],
        "moet_adamw_clipped": [A, i32, O, vp, vp, f64, vp, vp, vp, sz, vp],
        "moet_grad_norm": [A, i32, f64, vp, vp, vp, sz, vp],
    }
    for name, args in sigs.items():
        f = getattr(_c, name)
        f.argtypes = args
        f.restype = ctypes.c_int32


_declare()

_CODE_M = (torch.float8_e4m3fn, torch.uint8)
_CODE_V = (torch.float8_e5m2, torch.uint8)
_EITHER = (torch.bfloat16, torch.float32)


def moet_workspace_size(p: Problem, stage: int) -> int:
    out = ctypes.c_size_t(0)
    status = _c.moet_workspace_size(ctypes.byref(p), int(stage), ctypes.byref(out))
    if status != _lib.MOE_OK:
        raise _lib.MoEError(status, "moet_workspace_size")
    return int(out.value)


# ---- rows sorted by expert and back

def moet_dispatch(p: Problem, topk_idx, weight, x, counts, offsets, perm, inv, x_perm, ws, stream=None):
    dev, R, n, dt = _device("topk_idx", topk_idx), p.T * p.k, p.T * p.d_model, _rows(p)
    _call(_c.moet_dispatch, dev, stream, ctypes.byref(p), _ptr("topk_idx", topk_idx, R, _I32, dev),
          _opt("weight", weight, R, _F32, dev), _ptr("x", x, n, dt, dev), _ptr("counts", counts, p.E, _I32, dev),
          _ptr("offsets", offsets, p.E + 1, _I32, dev), _ptr("perm", perm, R, _I32, dev), _ptr("inv", inv, R, _I32, dev),
          _ptr("x_perm", x_perm, n * p.k, dt, dev), *_ws(ws, dev))


def moet_dispatch_backward(p: Problem, dx_perm, inv, x, weight, residual, dx, dweight, stream=None):
    dev, R, n, dt = _device("dx_perm", dx_perm), p.T * p.k, p.T * p.d_model, _rows(p)
    _call(_c.moet_dispatch_backward, dev, stream, ctypes.byref(p), _ptr("dx_perm", dx_perm, n * p.k, dt, dev),
          _ptr("inv", inv, R, _I32, dev), _opt("x", x, n, dt, dev), _opt("weight", weight, R, _F32, dev),
          _opt("residual", residual, n, dt, dev), _ptr("dx", dx, n, dt, dev), _opt("dweight", dweight, R, _F32, dev))


def moet_combine(p: Problem, y_perm, inv, gate, residual, y, stream=None):
    dev, R, n, dt = _device("y_perm", y_perm), p.T * p.k, p.T * p.d_model, _rows(p)
    _call(_c.moet_combine, dev, stream, ctypes.byref(p), _ptr("y_perm", y_perm, n * p.k, dt, dev),
          _ptr("inv", inv, R, _I32, dev), _opt("gate", gate, R, _F32, dev), _opt("residual", residual, n, dt, dev),
          _ptr("y", y, n, dt, dev))


def moet_combine_backward(p: Problem, dy, inv, y_perm, gate, dy_perm, dgate, stream=None):
    dev, R, n, dt = _device("dy", dy), p.T * p.k, p.T * p.d_model, _rows(p)
    _call(_c.moet_combine_backward, dev, stream, ctypes.byref(p), _ptr("dy", dy, n, dt, dev),
          _ptr("inv", inv, R, _I32, dev), _opt("y_perm", y_perm, n * p.k, dt, dev), _opt("gate", gate, R, _F32, dev),
          _ptr("dy_perm", dy_perm, n * p.k, dt, dev), _opt("dgate", dgate, R, _F32, dev))


def moet_gate_backward(p: Problem, logits, topk_idx, dgate, add, dlogits, stream=None):
    dev, R, n = _device("logits", logits), p.T * p.k, p.T * p.E
    _call(_c.moet_gate_backward, dev, stream, ctypes.byref(p), _ptr("logits", logits, n, _F32, dev),
          _ptr("topk_idx", topk_idx, R, _I32, dev), _ptr("dgate", dgate, R, _F32, dev), _opt("add", add, n, _F32, dev),
          _ptr("dlogits", dlogits, n, _F32, dev))


# ---- a dense projection

def moet_linear(p: Problem, x, W, bias, act, residual, u, y, ws, stream=None):
    dev, T, K, N = _device("x", x), p.T, p.d_model, p.d_expert
    _call(_c.moet_linear, dev, stream, ctypes.byref(p), _ptr("x", x, T * K, _BF16, dev), _ptr("W", W, K * N, _BF16, dev),
          _opt("bias", bias, N, _BF16, dev), act, _opt("residual", residual, T * N, _BF16, dev),
          _opt("u", u, T * N, _BF16, dev), _ptr("y", y, T * N, _BF16, dev), *_ws(ws, dev))


def moet_linear_backward(p: Problem, x, W, u, act, dy, dx, dW, dbias, ws, stream=None):
    dev, T, K, N = _device("dy", dy), p.T, p.d_model, p.d_expert
    _call(_c.moet_linear_backward, dev, stream, ctypes.byref(p), _opt("x", x, T * K, _BF16, dev),
          _opt("W", W, K * N, _BF16, dev), _opt("u", u, T * N, _BF16, dev), act, _ptr("dy", dy, T * N, _BF16, dev),
          _opt("dx", dx, T * K, _BF16, dev), _opt("dW", dW, K * N, _BF16, dev), _opt("dbias", dbias, N, _BF16, dev),
          *_ws(ws, dev))


# ---- the optimizer's step

def _dtype_of(name, t):
    if t.dtype == torch.bfloat16:
        return MOE_DTYPE_BF16
    if t.dtype == torch.float32:
        return MOE_DTYPE_F32
    raise TypeError(f"{name} has type {t.dtype}, expected {torch.bfloat16} or {torch.float32}")


def set_grad(e: Tensor, grad, dev, name="grad"):
    """Gives an entry its gradient."""
    e.grad = _ptr(name, grad, e.n, _EITHER, dev)
    e.grad_dtype = MOE_DTYPE_BF16 if grad.dtype == torch.bfloat16 else MOE_DTYPE_F32


def tensor_entry(param, grad, master, m, m_scale, v, v_scale, lr_factor=1.0, weight_decay=0.0) -> Tensor:
    """The entry of a parameter: bfloat16 with a float32 master copy, or float32 without. Moments
    are float32, or with scales e4m3 and e5m2 codes. grad may be None and given later (set_grad)."""
    dev = _device("param", param)
    n, small = param.numel(), m_scale is not None
    blocks = (n + 127) // 128
    e = Tensor(n=n, param_dtype=_dtype_of("param", param), lr_factor=lr_factor, weight_decay=weight_decay)
    if (param.dtype == torch.bfloat16) != (master is not None):
        raise ValueError("a bfloat16 parameter has a float32 master copy, a float32 one none")
    e.param = _ptr("param", param, n, _EITHER, dev)
    e.master = _opt("master", master, n, _F32, dev)
    e.m = _ptr("m", m, n, _CODE_M if small else _F32, dev)
    e.v = _ptr("v", v, n, _CODE_V if small else _F32, dev)
    e.m_scale = _ptr("m_scale", m_scale, blocks, _ext._SCALE, dev) if small else None
    e.v_scale = _ptr("v_scale", v_scale, blocks, _ext._SCALE, dev) if small else None
    if grad is not None:
        set_grad(e, grad, dev)
    return e


def _list(tensors):
    """(array, count) of a ctypes array or a sequence of entries."""
    if isinstance(tensors, ctypes.Array):
        return tensors, len(tensors)
    return (Tensor * max(1, len(tensors)))(*tensors), len(tensors)


def moet_adamw(tensors, opt: AdamWOptions, counter, lr_scale, grad_scale, stream=None):
    dev = _device("counter", counter)
    arr, count = _list(tensors)
    _call(_c.moet_adamw, dev, stream, arr, count, ctypes.byref(opt), _ptr("counter", counter, 2, _I32, dev),
          _opt("lr_scale", lr_scale, 1, _F32, dev), _opt("grad_scale", grad_scale, 1, _F32, dev))


def moet_grad_norm(tensors, max_norm, norm, scale, ws, stream=None):
    dev = _device("norm", norm)
    arr, count = _list(tensors)
    _call(_c.moet_grad_norm, dev, stream, arr, count, max_norm, _ptr("norm", norm, 1, _F32, dev),
          _opt("scale", scale, 1, _F32, dev), *_ws(ws, dev))


def moet_adamw_clipped(tensors, opt: AdamWOptions, counter, lr_scale, max_norm, norm, scale, ws, stream=None):
    dev = _device("counter", counter)
    arr, count = _list(tensors)
    _call(_c.moet_adamw_clipped, dev, stream, arr, count, ctypes.byref(opt), _ptr("counter", counter, 2, _I32, dev),
          _opt("lr_scale", lr_scale, 1, _F32, dev), max_norm, _ptr("norm", norm, 1, _F32, dev),
          _opt("scale", scale, 1, _F32, dev), *_ws(ws, dev))
