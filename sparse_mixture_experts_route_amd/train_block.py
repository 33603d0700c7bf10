"""A block that trains: norm with residual, the routed experts, a dense expert beside
them, their gradients, the balance loss and the optimizer's step, for a fixed shape."""

from __future__ import annotations

from typing import Dict, Optional

import torch

from . import _ext, _lib, _train
from .layer import _torch_stream
from .optim import AdamW

_BF = torch.bfloat16


class MoETrainBlock:
    """RMS norm, routed experts and (when V1 is given) a dense expert, with residual:

      h = x + residual,  n = rmsnorm(h) gain
      y = routed(n) + (GELU(n V1 + c1) V2 + c2)

    params, by name: gain [d_model], w_router [d_model, E], W1 [E, d_model, d_expert],
    W2 [E, d_expert, d_model] bfloat16; router_bias [E] float32, optional; the dense
    expert's V1 [d_model, D], c1 [D], V2 [D, d_model], c2 [d_model] bfloat16, all or none.
    The tensors are used and updated in place. `coef` weighs the balance loss. The
    optimizer's arguments are AdamW's (decay: of weights of two or more dimensions).

    A step is forward, backward with the gradient of y (and of h, where the residual
    stream goes on), and step. Gradients are in `grads`, the balance loss in `loss`. The
    layer's limits for training hold: E a multiple of 8, k <= 8. All calls work in this
    object's buffers: one stream at a time, and calls on different streams are ordered
    by the caller. The buffers' memory is not handed out again while work of a torch
    stream is in flight on it; for a raw stream handle the caller keeps the object until
    that work has ended. x, residual and dy are kept by the caller until the backward
    pass has ended; it may be called again, with another dy, before the next step.
    """

    def __init__(self, T: int, d_model: int, E: int, k: int, d_expert: int, params: Dict[str, torch.Tensor],
                 coef: float = 0.01, eps: float = 1e-6, weight_decay: float = 0.01, stream=None, **optimizer):
        names = ["gain", "w_router", "W1", "W2"]
        dense = [n for n in ("V1", "c1", "V2", "c2") if params.get(n) is not None]
        if len(dense) not in (0, 4):
            raise ValueError("a dense expert has V1, c1, V2 and c2")
        bias = params.get("router_bias") is not None
        self.names = names + (["router_bias"] if bias else []) + dense
        for n in self.names[:4]:
            if params.get(n) is None:
                raise ValueError(f"params lack {n}")
        unknown = [n for n in params if params[n] is not None and n not in self.names]
        if unknown:
            raise ValueError(f"params have unknown names: {', '.join(unknown)}")
        self.params = {n: params[n] for n in self.names}
        self.coef, self.eps = float(coef), float(eps)
        self.problem = p = _lib.make_problem(T, d_model, E, k, d_expert, _BF)
        D = params["V2"].shape[0] if dense else 0
        sizes = {"gain": d_model, "w_router": d_model * E, "W1": E * d_model * d_expert, "W2": E * d_model * d_expert,
                 "router_bias": E, "V1": d_model * D, "c1": D, "V2": D * d_model, "c2": d_model}
        self.index = index = _ext._device("gain", params["gain"])
        dev = torch.device("cuda", index)
        for n in self.names:
            _ext._ptr(n, self.params[n], sizes[n], (torch.float32,) if n == "router_bias" else (_BF,), index)

        def new(shape, dtype=_BF):
            return torch.empty(shape, dtype=dtype, device=dev)

        def space(size):
            return new((size,), torch.uint8)

        self._known = {_ext._handle(index, stream)}
        # allocated for the stream that first writes them: what it did before with their memory is behind it
        with torch.cuda.stream(_torch_stream(dev, stream)):
            self.h, self.n, self.y, self.dn, self.dx = (new((T, d_model)) for _ in range(5))
            self.rstd = new((T,), torch.float32)
            self.loss, self.counts = new((1,), torch.float32), new((E,), torch.int32)
            self.grads = {n: torch.empty_like(self.params[n], dtype=torch.float32 if n == "gain" else None)
                          for n in self.names}
            self._ws = space(_ext.moex_workspace_size(p, _ext.MOEX_STAGE_TRAIN_BALANCED))
            self._ws_norm = space(_ext.moex_workspace_size(p, _ext.MOEX_STAGE_NORM_BACKWARD))
            self._dense = None
            if dense:
                up, down = _lib.make_problem(T, d_model, 1, 1, D, _BF), _lib.make_problem(T, D, 1, 1, d_model, _BF)
                self._dense = (up, down)
                self.u, self.a, self.da = (new((T, D)) for _ in range(3))
                self.routed, self.dn_dense, self.dn_both = (new((T, d_model)) for _ in range(3))
                self._same = torch.arange(T, dtype=torch.int32, device=dev)
                self._ws_dense = space(max(_train.moet_workspace_size(q, s) for q in (up, down) for s in
                                           (_train.MOET_STAGE_LINEAR, _train.MOET_STAGE_LINEAR_BACKWARD)))
            decay = [weight_decay if self.params[n].dim() > 1 else 0.0 for n in self.names]
            self.optimizer = AdamW([self.params[n] for n in self.names], weight_decay=decay, **optimizer)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(dev).synchronize()
        self._input = None

    def _keep(self, stream):
        """Tells the allocator, once for each, of the torch streams that use the buffers besides their own."""
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            return
        handle = _ext._handle(self.index, stream)
        if handle in self._known:
            return
        self._known.add(handle)
        s = _torch_stream(torch.device("cuda", self.index), stream)
        for t in (*vars(self).values(), *self.grads.values()):
            if isinstance(t, torch.Tensor):
                t.record_stream(s)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, stream=None):
        """(y, h): the block's output, and the stream it is to be added to (x itself without residual)."""
        p, w = self.problem, self.params
        self._keep(stream)
        self._input = x if residual is None else self.h
        _ext.moex_add_rmsnorm(p, x, residual, w["gain"], self.eps, None if residual is None else self.h, self.n, None, None,
                              self.rstd, stream)
        routed = self.y if self._dense is None else self.routed
        with torch.cuda.device(self.index):
            _lib.moe_forward_train(p, self.n, w["w_router"], w.get("router_bias"), w["W1"], w["W2"], routed, self._ws,
                                   _ext._handle(self.index, stream))
        if self._dense is not None:
            up, down = self._dense
            _train.moet_linear(up, self.n, w["V1"], w["c1"], _train.MOET_ACT_GELU, None, self.u, self.a, self._ws_dense, stream)
            _train.moet_linear(down, self.a, w["V2"], w["c2"], _train.MOET_ACT_NONE, routed, None, self.y, self._ws_dense,
                               stream)
        return self.y, self._input

    def backward(self, dy: torch.Tensor, dh: Optional[torch.Tensor] = None, token_mask: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """The gradient of x, and equal to it of the residual, for the last forward call; token_mask as the
        balance loss takes it."""
        if self._input is None:
            raise RuntimeError("backward without a forward call")
        p, w, g = self.problem, self.params, self.grads
        self._keep(stream)
        _ext.moex_backward_balanced(p, self.n, w["w_router"], w["W1"], w["W2"], dy, token_mask, self.coef, self.dn,
                                    g["w_router"], g.get("router_bias"), g["W1"], g["W2"], self.loss, self.counts, None,
                                    self._ws, stream)
        dn = self.dn
        if self._dense is not None:
            up, down = self._dense
            _train.moet_linear_backward(down, self.a, w["V2"], None, _train.MOET_ACT_NONE, dy, self.da, g["V2"], g["c2"],
                                        self._ws_dense, stream)
            _train.moet_linear_backward(up, self.n, w["V1"], self.u, _train.MOET_ACT_GELU, self.da, self.dn_dense, g["V1"],
                                        g["c1"], self._ws_dense, stream)
            dn = self.dn_both  # the two paths' gradients of n, added: one row a token, in its place
            one = _lib.make_problem(p.T, p.d_model, 1, 1, 64, _BF)
            _train.moet_combine(one, self.dn_dense, self._same, None, self.dn, dn, stream)
        _ext.moex_add_rmsnorm_backward(p, self._input, w["gain"], self.rstd, dn, dh, self.dx, g["gain"], self._ws_norm, stream)
        return self.dx

    def step(self, stream=None) -> Optional[torch.Tensor]:
        """Updates the parameters; the gradients' norm before clipping, None without max_norm."""
        return self.optimizer.step([self.grads[n] for n in self.names], stream)
