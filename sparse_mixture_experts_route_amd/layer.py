"""Convenience wrapper: buffers for one layer shape, allocated once with torch.

torch only provides device memory here; the forward itself is the library's
moe_forward (or the four stage entry points) on the current HIP stream, and for
the block with 8-bit experts moex_add_rmsnorm and moex_forward_fp8.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _ext, _lib


class MoEForward:
    """Holds outputs and workspace for a fixed (T, d_model, E, k, d_expert, dtype)."""

    def __init__(self, T: int, d_model: int, E: int, k: int, d_expert: int, dtype: torch.dtype,
                 device="cuda"):
        self.problem = _lib.make_problem(T, d_model, E, k, d_expert, dtype)
        self.dtype = dtype
        self.device = torch.device(device)
        ws_bytes = _lib.moe_workspace_size(self.problem, _lib.MOE_STAGE_FORWARD)
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device)
        self.y = torch.empty((T, d_model), dtype=dtype, device=self.device)

    def __call__(self, x: torch.Tensor, w_router: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                 router_bias: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        _lib.moe_forward(self.problem, x, w_router, router_bias, W1, W2, self.y, self.ws, stream)
        return self.y

    def stages(self, x, w_router, W1, W2, router_bias=None, stream=None, logits=True):
        """Run the four stage entry points one after another; return every intermediate.

        Routing goes through moe_route_ws, the router moe_forward runs, so both
        paths select on logits summed in the same order."""
        p = self.problem
        T, E, k = p.T, p.E, p.k
        R = T * k
        dev = self.device
        out = {
            "logits": torch.empty((T, E), dtype=torch.float32, device=dev) if logits else None,
            "idx": torch.empty((T, k), dtype=torch.int32, device=dev),
            "gate": torch.empty((T, k), dtype=torch.float32, device=dev),
            "counts": torch.empty(E, dtype=torch.int32, device=dev),
            "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "perm": torch.empty(R, dtype=torch.int32, device=dev),
            "inv": torch.empty(R, dtype=torch.int32, device=dev),
            "x_perm": torch.empty((R, p.d_model), dtype=self.dtype, device=dev),
            "y_perm": torch.empty((R, p.d_model), dtype=self.dtype, device=dev),
            "y": torch.empty((T, p.d_model), dtype=self.dtype, device=dev),
        }
        ws_p = torch.empty(_lib.moe_workspace_size(p, _lib.MOE_STAGE_PERMUTE), dtype=torch.uint8, device=dev)
        ws_f = torch.empty(_lib.moe_workspace_size(p, _lib.MOE_STAGE_GROUPED_FFN), dtype=torch.uint8, device=dev)
        ws_r = torch.empty(_lib.moe_workspace_size(p, _lib.MOE_STAGE_ROUTE), dtype=torch.uint8, device=dev)
        _lib.moe_route_ws(p, x, w_router, router_bias, out["logits"], out["idx"], out["gate"], ws_r, stream)
        _lib.moe_permute(p, out["idx"], x, out["counts"], out["offsets"], out["perm"], out["inv"], out["x_perm"],
                         ws_p, stream)
        _lib.moe_grouped_ffn(p, out["x_perm"], out["offsets"], W1, W2, out["y_perm"], ws_f, stream)
        _lib.moe_combine(p, out["y_perm"], out["inv"], out["gate"], out["y"], stream)
        return out


def _torch_stream(dev, stream):
    """`stream` (None: the current one, a torch stream or a HIP handle) as a torch stream of GPU dev."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if stream is None:
        return torch.cuda.current_stream(dev)
    return torch.cuda.ExternalStream(int(stream), dev) if int(stream) else torch.cuda.default_stream(dev)


class MoEBlockFP8:
    """RMS norm with residual and the layer with 8-bit experts, for a fixed shape.

    The expert weights are quantised once, here, and that is waited for: the
    object is ready for calls on any stream. A call adds x to the residual
    stream, norms it, routes on the 16-bit rows and runs the experts on the 8-bit
    ones; y and h (the stream after the addition) are this object's buffers, so a
    residual or x may be another block's h but not, with a residual, this one's
    (refused: outputs overlap no input).

    All calls work in the same buffers: one object serves one stream at a time, and
    calls on different streams are ordered by the caller. The buffers' memory is not
    handed out again while work of a torch stream is in flight on it; for a raw
    stream handle the caller keeps the object until that work has ended.
    """

    def __init__(self, T: int, d_model: int, E: int, k: int, d_expert: int, gain: torch.Tensor,
                 w_router: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                 router_bias: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None):
        self.problem = p = _lib.make_problem(T, d_model, E, k, d_expert, torch.bfloat16)
        self.gain, self.w_router, self.router_bias, self.eps = gain, w_router, router_bias, eps
        dev = torch.device("cuda", _ext._device("W1", W1))
        self._known = {_ext._handle(dev.index, stream)}  # streams that the allocator knows to use the buffers

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=dev)

        # allocated for the stream that first writes them: what it did before with their memory is behind it
        with torch.cuda.stream(_torch_stream(dev, stream)):
            self.experts = [new(s, torch.uint8) for s in _ext.expert_shapes(p)]
            _ext.moex_quantize_experts(p, W1, W2, *self.experts, None)
            self.ws = new((_ext.moex_workspace_size(p, _ext.MOEX_STAGE_FORWARD_FP8),), torch.uint8)
            self.h, self.normed, self.y = (new((T, d_model), torch.bfloat16) for _ in range(3))
            self.x8 = new((T, _ext.code_pitch(d_model)), torch.float8_e4m3fn)
            self.x_scale = new((T, _ext.scale_pitch(d_model)), torch.uint8)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(dev).synchronize()

    def _keep(self, stream):
        """Tells the allocator, once for each, of the torch streams that use the buffers besides their own."""
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            return
        dev = self.y.device
        handle = _ext._handle(dev.index, stream)
        if handle not in self._known:
            self._known.add(handle)
            s = _torch_stream(dev, stream)
            for t in (*self.experts, self.ws, self.h, self.normed, self.y, self.x8, self.x_scale):
                t.record_stream(s)

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, stream=None):
        """(y, h): the layer's output, and the stream it is to be added to (x itself without residual)."""
        p, h = self.problem, self.h if residual is not None else None
        self._keep(stream)
        _ext.moex_add_rmsnorm(p, x, residual, self.gain, self.eps, h, self.normed, self.x8, self.x_scale, None, stream)
        _ext.moex_forward_fp8(p, self.normed, self.x8, self.x_scale, self.w_router, self.router_bias, *self.experts,
                              self.y, self.ws, stream)
        return self.y, h if h is not None else x
