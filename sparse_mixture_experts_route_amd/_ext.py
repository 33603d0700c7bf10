"""The operators around the layer (include/moe_ext.h): argument marshalling.

The functions carry the C names and argument order. Unlike the layer's own
calls they also check each tensor's type and size against the problem, and run
on the device that holds the tensors: its current stream is used unless one is
given.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MOE_DTYPE_BF16, Problem

MOEX_STAGE_NORM_BACKWARD = 0
MOEX_STAGE_BALANCE = 1
MOEX_STAGE_FFN_FP8 = 2
MOEX_STAGE_FORWARD_FP8 = 3
MOEX_STAGE_TRAIN_BALANCED = 4

_c = _lib.raw_lib()


def _declare():
    P = ctypes.POINTER(Problem)
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    sigs = {
        "moex_workspace_size": [P, i32, ctypes.POINTER(sz)],
        "moex_add_rmsnorm": [P, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp],
        "moex_add_rmsnorm_backward": [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moex_quantize_rows": [P, vp, vp, vp, vp],
        "moex_balance_loss": [P, vp, vp, vp, f32, vp, vp, vp, vp, vp, sz, vp],
        "moex_backward_balanced": [P, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moex_quantize_experts": [P, vp, vp, vp, vp, vp, vp, vp],
        "moex_grouped_ffn_fp8": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moex_forward_fp8": [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
    }
    for name, args in sigs.items():
        f = getattr(_c, name)
        f.argtypes = args
        f.restype = ctypes.c_int32


_declare()

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_BF16 = (torch.bfloat16,)
_BYTE = (torch.uint8, torch.bool)
_CODE = (torch.uint8, torch.float8_e4m3fn)
_SCALE = (torch.uint8, torch.float8_e8m0fnu)


def code_pitch(K: int) -> int:
    """Bytes of one row's e4m3 codes for K values."""
    return (int(K) + 127) // 128 * 128


def scale_pitch(K: int) -> int:
    """Bytes of one row's scales for K values."""
    return (int(K) + 2047) // 2048 * 16


class _Args:
    """Checks tensors against what a call expects and finds the device they share."""

    __slots__ = ("where", "device")

    def __init__(self, where: str):
        self.where = where
        self.device = None

    def __call__(self, name, t, n, dtypes, required=True):
        if t is None:
            if required:
                raise ValueError(f"{self.where}: {name} is required")
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: {name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{self.where}: {name} must live on the GPU")
        if t.dtype not in dtypes:
            raise TypeError(f"{self.where}: {name} has type {t.dtype}, expected {dtypes[0]}")
        if t.numel() != n:
            raise ValueError(f"{self.where}: {name} holds {t.numel()} values, expected {n}")
        if not t.is_contiguous():
            raise ValueError(f"{self.where}: {name} must be contiguous")
        if self.device is None:
            self.device = t.device
        elif t.device != self.device:
            raise ValueError(f"{self.where}: {name} is on {t.device}, other arguments on {self.device}")
        return t.data_ptr()

    def ws(self, t):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: ws must be a torch.Tensor")
        return self("ws", t, t.numel(), (t.dtype,)), t.numel() * t.element_size()

    def call(self, stream, *args):
        f = getattr(_c, self.where)
        dev = self.device
        if stream is None:
            stream = torch.cuda.current_stream(dev).cuda_stream
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device != dev:
                raise ValueError(f"{self.where}: the stream is on {stream.device}, the tensors on {dev}")
            stream = stream.cuda_stream
        if dev.index == torch.cuda.current_device():
            status = f(*args, int(stream))
        else:
            with torch.cuda.device(dev):
                status = f(*args, int(stream))
        if status != _lib.MOE_OK:
            raise _lib.MoEError(status, self.where)


def _rows(p: Problem):
    return _BF16 if p.dtype == MOE_DTYPE_BF16 else _F32


def moex_workspace_size(p: Problem, stage: int) -> int:
    out = ctypes.c_size_t(0)
    status = _c.moex_workspace_size(ctypes.byref(p), int(stage), ctypes.byref(out))
    if status != _lib.MOE_OK:
        raise _lib.MoEError(status, "moex_workspace_size")
    return int(out.value)


def moex_add_rmsnorm(p: Problem, x, residual, gain, eps, h, y, y8, y_scale, rstd, stream=None):
    a, n, dt = _Args("moex_add_rmsnorm"), p.T * p.d_model, _rows(p)
    args = (ctypes.byref(p), a("x", x, n, dt), a("residual", residual, n, dt, False), a("gain", gain, p.d_model, dt),
            float(eps), a("h", h, n, dt, False), a("y", y, n, dt, False),
            a("y8", y8, p.T * code_pitch(p.d_model), _CODE, False),
            a("y_scale", y_scale, p.T * scale_pitch(p.d_model), _SCALE, False), a("rstd", rstd, p.T, _F32, False))
    a.call(stream, *args)


def moex_add_rmsnorm_backward(p: Problem, h, gain, rstd, dy, dh, dx, dgain, ws, stream=None):
    a, n, dt = _Args("moex_add_rmsnorm_backward"), p.T * p.d_model, _rows(p)
    args = (ctypes.byref(p), a("h", h, n, dt), a("gain", gain, p.d_model, dt), a("rstd", rstd, p.T, _F32),
            a("dy", dy, n, dt), a("dh", dh, n, dt, False), a("dx", dx, n, dt), a("dgain", dgain, p.d_model, _F32))
    a.call(stream, *args, *a.ws(ws))


def moex_quantize_rows(p: Problem, x, x8, x_scale, stream=None):
    a = _Args("moex_quantize_rows")
    args = (ctypes.byref(p), a("x", x, p.T * p.d_model, _rows(p)), a("x8", x8, p.T * code_pitch(p.d_model), _CODE),
            a("x_scale", x_scale, p.T * scale_pitch(p.d_model), _SCALE))
    a.call(stream, *args)


def moex_balance_loss(p: Problem, logits, topk_idx, token_mask, coef, loss, counts, mean_prob, dlogits, ws,
                      stream=None):
    a = _Args("moex_balance_loss")
    args = (ctypes.byref(p), a("logits", logits, p.T * p.E, _F32), a("topk_idx", topk_idx, p.T * p.k, _I32),
            a("token_mask", token_mask, p.T, _BYTE, False), float(coef), a("loss", loss, 1, _F32),
            a("counts", counts, p.E, _I32), a("mean_prob", mean_prob, p.E, _F32),
            a("dlogits", dlogits, p.T * p.E, _F32, False))
    a.call(stream, *args, *a.ws(ws))


def moex_backward_balanced(p: Problem, x, w_router, W1, W2, dy, token_mask, coef, dx, dw_router, dbias, dW1, dW2, loss,
                           counts, mean_prob, ws, stream=None):
    a, td, w = _Args("moex_backward_balanced"), p.T * p.d_model, p.E * p.d_model * p.d_expert
    args = (ctypes.byref(p), a("x", x, td, _BF16), a("w_router", w_router, p.d_model * p.E, _BF16),
            a("W1", W1, w, _BF16), a("W2", W2, w, _BF16), a("dy", dy, td, _BF16),
            a("token_mask", token_mask, p.T, _BYTE, False), float(coef), a("dx", dx, td, _BF16),
            a("dw_router", dw_router, p.d_model * p.E, _BF16), a("dbias", dbias, p.E, _F32, False),
            a("dW1", dW1, w, _BF16), a("dW2", dW2, w, _BF16), a("loss", loss, 1, _F32),
            a("counts", counts, p.E, _I32, False), a("mean_prob", mean_prob, p.E, _F32, False))
    a.call(stream, *args, *a.ws(ws))


def expert_shapes(p: Problem):
    """Shapes of the 8-bit expert weights (W1q, W1s, W2q, W2s), all one byte per value."""
    def shapes(K, N):
        kb = code_pitch(K) // 128
        return (p.E, N // 32, kb, 4, 2, 32, 16), (p.E, N // 32, kb, 32)
    return (*shapes(p.d_model, p.d_expert), *shapes(p.d_expert, p.d_model))


def _experts(a: _Args, p: Problem, W1q, W1s, W2q, W2s):
    n1, n2 = p.E * p.d_expert * code_pitch(p.d_model), p.E * p.d_model * code_pitch(p.d_expert)
    return (a("W1q", W1q, n1, _CODE), a("W1s", W1s, n1 // 128, _SCALE), a("W2q", W2q, n2, _CODE),
            a("W2s", W2s, n2 // 128, _SCALE))


def moex_quantize_experts(p: Problem, W1, W2, W1q, W1s, W2q, W2s, stream=None):
    a, w = _Args("moex_quantize_experts"), p.E * p.d_model * p.d_expert
    args = (ctypes.byref(p), a("W1", W1, w, _rows(p)), a("W2", W2, w, _rows(p)), *_experts(a, p, W1q, W1s, W2q, W2s))
    a.call(stream, *args)


def moex_grouped_ffn_fp8(p: Problem, x8, x_scale, perm, offsets, W1q, W1s, W2q, W2s, y_perm, ws, stream=None):
    a, R = _Args("moex_grouped_ffn_fp8"), p.T * p.k
    rows = p.T if perm is not None else R
    args = (ctypes.byref(p), a("x8", x8, rows * code_pitch(p.d_model), _CODE),
            a("x_scale", x_scale, rows * scale_pitch(p.d_model), _SCALE), a("perm", perm, R, _I32, False),
            a("offsets", offsets, p.E + 1, _I32), *_experts(a, p, W1q, W1s, W2q, W2s),
            a("y_perm", y_perm, R * p.d_model, _BF16))
    a.call(stream, *args, *a.ws(ws))


def moex_forward_fp8(p: Problem, x, x8, x_scale, w_router, router_bias, W1q, W1s, W2q, W2s, y, ws, stream=None):
    a, td = _Args("moex_forward_fp8"), p.T * p.d_model
    args = (ctypes.byref(p), a("x", x, td, _BF16), a("x8", x8, p.T * code_pitch(p.d_model), _CODE, False),
            a("x_scale", x_scale, p.T * scale_pitch(p.d_model), _SCALE, False),
            a("w_router", w_router, p.d_model * p.E, _BF16), a("router_bias", router_bias, p.E, _F32, False),
            *_experts(a, p, W1q, W1s, W2q, W2s), a("y", y, td, _BF16))
    a.call(stream, *args, *a.ws(ws))
