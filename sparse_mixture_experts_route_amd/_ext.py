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


def _ptr(name, t, n, dtypes, dev):
    """Address of a tensor of n values of one of dtypes on GPU dev."""
    try:
        if t.get_device() == dev and t.dtype in dtypes and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise _refusal(name, t, n, dtypes, dev)


def _opt(name, t, n, dtypes, dev):
    """The same, or NULL for None."""
    return None if t is None else _ptr(name, t, n, dtypes, dev)


def _refusal(name, t, n, dtypes, dev):
    if t is None:
        return ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        return ValueError(f"{name} must live on the GPU")
    if t.dtype not in dtypes:
        return TypeError(f"{name} has type {t.dtype}, expected {dtypes[0]}")
    if t.numel() != n:
        return ValueError(f"{name} holds {t.numel()} values, expected {n}")
    if not t.is_contiguous():
        return ValueError(f"{name} must be contiguous")
    return ValueError(f"{name} is on {t.device}, other arguments on GPU {dev}")


def _device(name, t):
    """GPU of the first tensor of a call, which all others have to share."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise _refusal(name, t, 0, (), -1)
    return t.get_device()


def _ws(ws, dev):
    if not isinstance(ws, torch.Tensor):
        raise _refusal("ws", ws, 0, (), dev)
    return _ptr("ws", ws, ws.numel(), (ws.dtype,), dev), ws.numel() * ws.element_size()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# without the initialisation check of torch.cuda.current_device: a call holds a GPU tensor by then
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _handle(dev, stream):
    """HIP handle of `stream` (None: GPU dev's current stream)."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on GPU {dev}")
        return stream.cuda_stream
    return int(stream)


def _call(f, dev, stream, *args):
    """Calls f on GPU dev and on `stream` (None: that GPU's current stream)."""
    stream = _handle(dev, stream)
    if dev == _current_device():
        status = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args, stream)
    if status != _lib.MOE_OK:
        raise _lib.MoEError(status, f.__name__)


def _rows(p: Problem):
    return _BF16 if p.dtype == MOE_DTYPE_BF16 else _F32


def moex_workspace_size(p: Problem, stage: int) -> int:
    out = ctypes.c_size_t(0)
    status = _c.moex_workspace_size(ctypes.byref(p), int(stage), ctypes.byref(out))
    if status != _lib.MOE_OK:
        raise _lib.MoEError(status, "moex_workspace_size")
    return int(out.value)


def moex_add_rmsnorm(p: Problem, x, residual, gain, eps, h, y, y8, y_scale, rstd, stream=None):
    dev, T, d, dt = _device("x", x), p.T, p.d_model, _rows(p)
    n = T * d
    _call(_c.moex_add_rmsnorm, dev, stream, ctypes.byref(p), _ptr("x", x, n, dt, dev),
          _opt("residual", residual, n, dt, dev), _ptr("gain", gain, d, dt, dev), eps, _opt("h", h, n, dt, dev),
          _opt("y", y, n, dt, dev), _opt("y8", y8, T * code_pitch(d), _CODE, dev),
          _opt("y_scale", y_scale, T * scale_pitch(d), _SCALE, dev), _opt("rstd", rstd, T, _F32, dev))


def moex_add_rmsnorm_backward(p: Problem, h, gain, rstd, dy, dh, dx, dgain, ws, stream=None):
    dev, T, d, dt = _device("h", h), p.T, p.d_model, _rows(p)
    n = T * d
    _call(_c.moex_add_rmsnorm_backward, dev, stream, ctypes.byref(p), _ptr("h", h, n, dt, dev),
          _ptr("gain", gain, d, dt, dev), _ptr("rstd", rstd, T, _F32, dev), _ptr("dy", dy, n, dt, dev),
          _opt("dh", dh, n, dt, dev), _ptr("dx", dx, n, dt, dev), _ptr("dgain", dgain, d, _F32, dev), *_ws(ws, dev))


def moex_quantize_rows(p: Problem, x, x8, x_scale, stream=None):
    dev, T, d = _device("x", x), p.T, p.d_model
    _call(_c.moex_quantize_rows, dev, stream, ctypes.byref(p), _ptr("x", x, T * d, _rows(p), dev),
          _ptr("x8", x8, T * code_pitch(d), _CODE, dev), _ptr("x_scale", x_scale, T * scale_pitch(d), _SCALE, dev))


def moex_balance_loss(p: Problem, logits, topk_idx, token_mask, coef, loss, counts, mean_prob, dlogits, ws,
                      stream=None):
    dev, T, E = _device("logits", logits), p.T, p.E
    _call(_c.moex_balance_loss, dev, stream, ctypes.byref(p), _ptr("logits", logits, T * E, _F32, dev),
          _ptr("topk_idx", topk_idx, T * p.k, _I32, dev), _opt("token_mask", token_mask, T, _BYTE, dev), coef,
          _ptr("loss", loss, 1, _F32, dev), _ptr("counts", counts, E, _I32, dev),
          _ptr("mean_prob", mean_prob, E, _F32, dev), _opt("dlogits", dlogits, T * E, _F32, dev), *_ws(ws, dev))


def moex_backward_balanced(p: Problem, x, w_router, W1, W2, dy, token_mask, coef, dx, dw_router, dbias, dW1, dW2, loss,
                           counts, mean_prob, ws, stream=None):
    dev, T, d, E = _device("x", x), p.T, p.d_model, p.E
    td, w = T * d, E * d * p.d_expert
    _call(_c.moex_backward_balanced, dev, stream, ctypes.byref(p), _ptr("x", x, td, _BF16, dev),
          _ptr("w_router", w_router, d * E, _BF16, dev), _ptr("W1", W1, w, _BF16, dev), _ptr("W2", W2, w, _BF16, dev),
          _ptr("dy", dy, td, _BF16, dev), _opt("token_mask", token_mask, T, _BYTE, dev), coef,
          _ptr("dx", dx, td, _BF16, dev), _ptr("dw_router", dw_router, d * E, _BF16, dev),
          _opt("dbias", dbias, E, _F32, dev), _ptr("dW1", dW1, w, _BF16, dev), _ptr("dW2", dW2, w, _BF16, dev),
          _ptr("loss", loss, 1, _F32, dev), _opt("counts", counts, E, _I32, dev),
          _opt("mean_prob", mean_prob, E, _F32, dev), *_ws(ws, dev))


def expert_shapes(p: Problem):
    """Shapes of the 8-bit expert weights (W1q, W1s, W2q, W2s), all one byte per value."""
    def shapes(K, N):
        kb = code_pitch(K) // 128
        return (p.E, N // 32, kb, 4, 2, 32, 16), (p.E, N // 32, kb, 32)
    return (*shapes(p.d_model, p.d_expert), *shapes(p.d_expert, p.d_model))


def _experts(p: Problem, W1q, W1s, W2q, W2s, dev):
    n1, n2 = p.E * p.d_expert * code_pitch(p.d_model), p.E * p.d_model * code_pitch(p.d_expert)
    return (_ptr("W1q", W1q, n1, _CODE, dev), _ptr("W1s", W1s, n1 // 128, _SCALE, dev),
            _ptr("W2q", W2q, n2, _CODE, dev), _ptr("W2s", W2s, n2 // 128, _SCALE, dev))


def moex_quantize_experts(p: Problem, W1, W2, W1q, W1s, W2q, W2s, stream=None):
    dev, w = _device("W1", W1), p.E * p.d_model * p.d_expert
    _call(_c.moex_quantize_experts, dev, stream, ctypes.byref(p), _ptr("W1", W1, w, _rows(p), dev),
          _ptr("W2", W2, w, _rows(p), dev), *_experts(p, W1q, W1s, W2q, W2s, dev))


def moex_grouped_ffn_fp8(p: Problem, x8, x_scale, perm, offsets, W1q, W1s, W2q, W2s, y_perm, ws, stream=None):
    dev, d, R = _device("x8", x8), p.d_model, p.T * p.k
    rows = R if perm is None else p.T
    _call(_c.moex_grouped_ffn_fp8, dev, stream, ctypes.byref(p), _ptr("x8", x8, rows * code_pitch(d), _CODE, dev),
          _ptr("x_scale", x_scale, rows * scale_pitch(d), _SCALE, dev), _opt("perm", perm, R, _I32, dev),
          _ptr("offsets", offsets, p.E + 1, _I32, dev), *_experts(p, W1q, W1s, W2q, W2s, dev),
          _ptr("y_perm", y_perm, R * d, _BF16, dev), *_ws(ws, dev))


def moex_forward_fp8(p: Problem, x, x8, x_scale, w_router, router_bias, W1q, W1s, W2q, W2s, y, ws, stream=None):
    dev, T, d, E = _device("x", x), p.T, p.d_model, p.E
    _call(_c.moex_forward_fp8, dev, stream, ctypes.byref(p), _ptr("x", x, T * d, _BF16, dev),
          _opt("x8", x8, T * code_pitch(d), _CODE, dev), _opt("x_scale", x_scale, T * scale_pitch(d), _SCALE, dev),
          _ptr("w_router", w_router, d * E, _BF16, dev), _opt("router_bias", router_bias, E, _F32, dev),
          *_experts(p, W1q, W1s, W2q, W2s, dev), _ptr("y", y, T * d, _BF16, dev), *_ws(ws, dev))
