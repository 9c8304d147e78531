"""The routed layer with what stands in front of it in a model's block: the
norm of the token rows, the selection of experts from router scores, and the
block's input kept in 8 bits between forward and backward.

    h      = norm(x)                                 normalise
    scores = the caller's router projection of h
    out    = layer(h; select(scores))                forward
    dh, dscores                                      backward
    dx     = the norm's backward of dh and of the projection's share    finish

The router projection stays with the caller (a plain matrix product of its
own weights); everything else of the path runs in the library's kernels.

With ``keep`` naming an 8-bit format, a block holds between forward and
backward the checkpoint of x (1.03 bytes an element), the scores, the ids and
the weights, and nothing of the layer: ``backward`` norms the checkpoint
again, repeats the layer's forward for the experts chosen before, and goes
back from there. Blocks that train one after another may then share a layer
workspace. Gradients are those of the kept values: the norm's statistics, h and
the layer's context are formed anew from the checkpoint, the selection is not.
With ``keep=None`` x and the layer's saved context stay as they are: x may not
be written to before ``finish``, and a forward or backward on the same layer
before this block's ``backward`` would replace the context, so that ``backward``
is refused then.

`layer` is a ``binding.Layer`` or an ``ep.ExpertParallelLayer``.
"""

from __future__ import annotations

from typing import Dict, Optional

import torch

from . import binding as B


class RoutedBlock:
    """One block's forward and backward, one pass at a time: normalise, forward, backward, finish.

    `select`: ``binding.make_select_cfg(...)``; `route_bias`: fp32 [E], ranks only; `norm_weight` and
    `norm_bias`: [H] or None; `kind`: "rms" or "layer"; `keep`: "e4m3", "int8" or None."""

    def __init__(self, layer, select: B.SelectCfg, norm_weight: Optional[torch.Tensor] = None,
                 norm_bias: Optional[torch.Tensor] = None, kind: str = "rms", eps: float = 1e-6,
                 route_bias: Optional[torch.Tensor] = None, keep: Optional[str] = "e4m3"):
        if kind not in B.NORM_KINDS:
            raise ValueError(f"kind: expected one of {sorted(B.NORM_KINDS)}, got {kind!r}")
        if keep is not None and keep not in B.CKPT_FORMATS:
            raise ValueError(f"keep: expected one of {sorted(B.CKPT_FORMATS)} or None, got {keep!r}")
        self.layer = layer
        self.select = select
        self.norm_weight = norm_weight
        self.norm_bias = norm_bias
        self.kind = kind
        self.eps = eps
        self.route_bias = route_bias
        self.keep = keep
        self._x = None      # x, or its checkpoint
        self._stats = None  # (mean, rstd) of what is kept
        self._route = None  # (scores, ids, weights)
        self._passes = 0    # of the layer, when its context was this block's (keep=None)
        self._stage = "normalise"  # the call that comes next

    def _expects(self, call: str) -> None:
        if self._stage != call:
            raise RuntimeError(f"{call} called where {self._stage} comes next")

    def normalise(self, x: torch.Tensor) -> torch.Tensor:
        """h = norm(x) [Q, H] bf16; begins a pass and drops an unfinished one."""
        h, mean, rstd, ckpt = B.norm_fwd(x, self.norm_weight, self.norm_bias, kind=self.kind, eps=self.eps, save=self.keep)
        self._x = x if ckpt is None else ckpt
        self._stats = (mean, rstd)
        self._route = None
        self._stage = "forward"
        return h

    def forward(self, h: torch.Tensor, scores: torch.Tensor, counts: Optional[torch.Tensor] = None,
                train: bool = True) -> torch.Tensor:
        """The layer's output [Q, H] for the experts that `scores` [Q, E] select; `counts` as in
        binding.router_select. train=False ends the pass here and keeps nothing."""
        self._expects("forward")
        ids, weights = B.router_select(scores, self.select, self.route_bias, counts=counts)
        out = self.layer.forward(ids, weights, h, save_for_backward=train and self.keep is None)
        if train:
            self._route = (scores, ids, weights)
            self._passes = getattr(self.layer, "passes", None)  # a layer of the caller's own need not count
            self._stage = "backward"
        else:
            self._x = self._stats = None
            self._stage = "normalise"
        return out

    def backward(self, grad_out: torch.Tensor, grads: Dict[str, torch.Tensor], accumulate: bool = False,
                 grad_scale: float = 1.0):
        """(grad_h [Q, H] through the layer, grad_scores [Q, E]); fills the layer's LoRA gradients."""
        self._expects("backward")
        if self.keep is None and getattr(self.layer, "passes", None) != self._passes:
            raise RuntimeError("the layer's saved context is no longer this pass's: another forward or backward ran on the "
                               "layer (blocks that share one need keep=\"e4m3\" or \"int8\")")
        scores, ids, weights = self._route
        if self.keep is not None:
            h, mean, rstd, _ = B.norm_fwd(self._x, self.norm_weight, self.norm_bias, kind=self.kind, eps=self.eps,
                                          dtype=grad_out.dtype)
            self._stats = (mean, rstd)
            self.layer.forward(ids, weights, h)
        grad_route = torch.empty(weights.shape, dtype=torch.float32, device=weights.device)
        grad_h = self.layer.backward(grad_out, grads, accumulate=accumulate, grad_scale=grad_scale, grad_route=grad_route)
        grad_scores = B.router_select_bwd(scores, self.select, ids, grad_route)
        self._route = None
        self._stage = "finish"
        return grad_h, grad_scores

    def finish(self, grad_h: torch.Tensor, grad_weight: Optional[torch.Tensor] = None,
               grad_bias: Optional[torch.Tensor] = None, accumulate: bool = False):
        """(grad_x, grad_weight, grad_bias) of the norm from the whole gradient of h, the layer's share
        plus the router projection's; ends the pass."""
        self._expects("finish")
        mean, rstd = self._stats
        if self.norm_bias is not None and self.norm_weight is None and grad_bias is None and not accumulate:
            grad_bias = torch.empty_like(self.norm_bias)  # without a weight, norm_bwd would take grad_h's type
        out = B.norm_bwd(grad_h, self._x, rstd, self.norm_weight, mean=mean, kind=self.kind,
                         bias_grad=self.norm_bias is not None, grad_weight=grad_weight, grad_bias=grad_bias,
                         accumulate=accumulate)
        self._x = self._stats = None
        self._stage = "normalise"
        return out
