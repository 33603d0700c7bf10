"""AdamW over a list of tensors, on the library's moet_adamw and moet_adamw_clipped."""

from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import _ext, _train
from ._lib import MOE_DTYPE_BF16, MOE_DTYPE_F32, MOE_ERR_INVALID_ARGUMENT, MoEError
from .layer import _torch_stream

_KINDS = ("master", "m", "m_scale", "v", "v_scale")


class AdamW:
    """The optimizer's state for a fixed list of parameters, and its step.

    Parameters are float32, or bfloat16 with a float32 master copy that this object
    holds. Moments are float32, or with bits=8 codes of 8 bits with a scale per 128
    values (tensors of fewer than `least` values keep 32 bits; bits may also be one
    number per parameter). lr_factor and weight_decay may be numbers or one per
    parameter. With max_norm the gradients are clipped to that norm, and a step
    whose gradients are not finite is left out altogether (max_norm=inf: that alone).

    A step only enqueues work: it can be captured into a graph. It reads lr when it
    is enqueued, and at every replay `lr_scale`, a float32 tensor of this object
    that a schedule may write; the number of steps is kept on the GPU (`counter`).

    The parameters are updated where they were when the object was made; a step
    refuses one that has been given other memory since (as `p.data = q` does).

    state: buffers to go on from, lists by the names master, m, m_scale, v, v_scale
    (None where a parameter has none) and counter, as `state` gives them; they are
    used in place. All calls of an object are on one stream, or ordered by the caller;
    it is ready for any stream when it has been made. Its own buffers' memory is not
    handed out again while work of a torch stream is in flight on it; for a raw stream
    handle the caller keeps the object until that work has ended.
    """

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, lr_factor=1.0, bits=32, least: int = 4096, max_norm: Optional[float] = None,
                 seed: int = 0, state: Optional[dict] = None):
        self.params = list(params)
        if not 1 <= len(self.params) <= _train.MOET_MAX_TENSORS:
            raise ValueError(f"{len(self.params)} parameters, expected 1 to {_train.MOET_MAX_TENSORS}")
        n = len(self.params)
        self.device = torch.device("cuda", _ext._device("param", self.params[0]))
        self.lr, self.betas, self.eps, self.seed, self.max_norm = lr, tuple(betas), eps, int(seed), max_norm
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive")

        def each(v, name):
            v = list(v) if isinstance(v, (list, tuple)) else [v] * n
            if len(v) != n:
                raise ValueError(f"{len(v)} values of {name} for {n} parameters")
            return v

        given, width = isinstance(bits, (list, tuple)), each(bits, "bits")
        if any(b not in (8, 32) for b in width):
            raise ValueError("moments are held in 8 or in 32 bits")
        width = [b if given or p.numel() >= least else 32 for b, p in zip(width, self.params)]
        if state is None:
            state = self._fresh(width)
        missing = [k for k in (*_KINDS, "counter") if k not in state]
        if missing or any(len(state[k]) != n for k in _KINDS):
            raise ValueError(f"state needs lists of {n} for {', '.join(_KINDS)}, and a counter")
        for k in _KINDS:
            setattr(self, k, tuple(state[k]))  # the list below has their addresses
        self.counter = state["counter"]
        self._list = (_train.Tensor * n)()
        for i, (d, f) in enumerate(zip(each(weight_decay, "weight_decay"), each(lr_factor, "lr_factor"))):
            if self.params[i].get_device() != self.device.index:
                raise ValueError(f"parameter {i} is on {self.params[i].device}, the first on {self.device}")
            if not (0 <= f < math.inf and 0 <= d < math.inf):
                raise ValueError(f"parameter {i} has lr_factor {f} and weight_decay {d}, expected finite numbers from 0 on")
            self._list[i] = _train.tensor_entry(self.params[i], None, self.master[i], self.m[i], self.m_scale[i],
                                                self.v[i], self.v_scale[i], float(f), float(d))
            if any((getattr(self._list[i], k) or 0) % 16 for k in ("param", *_KINDS)):
                raise MoEError(MOE_ERR_INVALID_ARGUMENT, f"AdamW: parameter {i} or its state is not aligned to 16 bytes")
        self._entries = list(self._list)  # each entry's own view of the array
        self._held = [t for k in _KINDS for t in getattr(self, k) if t is not None]
        self._places = [p.data_ptr() for p in self.params]
        self._sizes = [p.numel() for p in self.params]
        self._options = _train.AdamWOptions()
        with torch.cuda.device(self.device):
            self.lr_scale = torch.ones(1, device=self.device)
            self.norm, self.scale = (torch.ones(1, device=self.device) for _ in range(2))
            self._ws = torch.empty(_train.MOET_GRAD_NORM_WS_BYTES, dtype=torch.uint8, device=self.device)
        self._known = {_ext._handle(self.device.index, None)}  # streams that the allocator knows to use the buffers
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()

    def _keep(self, stream):
        """Tells the allocator, once for each, of the torch streams that use the buffers besides their own."""
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            return
        handle = _ext._handle(self.device.index, stream)
        if handle not in self._known:
            self._known.add(handle)
            s = _torch_stream(self.device, stream)
            for t in (self.counter, self.lr_scale, self.norm, self.scale, self._ws, *self._held):
                t.record_stream(s)

    def _fresh(self, width):
        s = {k: [] for k in _KINDS}
        for p, b in zip(self.params, width):
            s["master"].append(p.detach().float().reshape(-1).contiguous() if p.dtype == torch.bfloat16 else None)
            shape = (p.numel(),)
            for k, t in (("m", torch.float8_e4m3fn), ("v", torch.float8_e5m2)):
                codes = torch.zeros(shape, dtype=torch.uint8 if b == 8 else torch.float32, device=p.device)
                s[k].append(codes.view(t) if b == 8 else codes)
                # scales of zeros are the smallest, 2^-120
                s[k + "_scale"].append(torch.full(((p.numel() + 127) // 128,), 7, dtype=torch.uint8, device=p.device)
                                       if b == 8 else None)
        s["counter"] = torch.zeros(2, dtype=torch.int32, device=self.device)
        return s

    @property
    def state(self) -> dict:
        """The buffers themselves (clone them to keep them)."""
        return {**{k: list(getattr(self, k)) for k in _KINDS}, "counter": self.counter}

    def step(self, grads: Sequence[torch.Tensor], stream=None) -> Optional[torch.Tensor]:
        """One step with a gradient of each parameter, bfloat16 or float32. Returns the norm of the
        gradients before clipping (this object's buffer), None without max_norm."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        if list(map(torch.Tensor.data_ptr, self.params)) != self._places:
            raise RuntimeError("a parameter's memory is not the one that this object was made with")
        self._keep(stream)
        dev, ptr, either, bf16 = self.device.index, _ext._ptr, _train._EITHER, torch.bfloat16
        for e, n, g in zip(self._entries, self._sizes, grads):  # _train.set_grad's, without reading n from the entry
            e.grad = ptr("grad", g, n, either, dev)
            e.grad_dtype = MOE_DTYPE_BF16 if g.dtype is bf16 else MOE_DTYPE_F32
        opt, clip = self._options, self.max_norm is not None
        opt.lr, (opt.beta1, opt.beta2), opt.eps, opt.seed = self.lr, self.betas, self.eps, self.seed & 0xFFFFFFFF
        if not clip:
            _train.moet_adamw(self._list, opt, self.counter, self.lr_scale, None, stream)
            return None
        _train.moet_adamw_clipped(self._list, opt, self.counter, self.lr_scale, self.max_norm, self.norm, self.scale, self._ws,
                                  stream)
        return self.norm
