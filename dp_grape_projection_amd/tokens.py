"""The two ends of a language model around the private update step, as torch
modules and functions: the token embedding, whose table can take part in the
step of a GrapeOptimizer, and the losses against a [V, d] table (cross entropy,
and distillation from a teacher's top logits). All of it runs in libdpg's
kernels; this module only wires tensors to those calls.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import binding as _b


class TokenEmbedding(torch.nn.Module):
    """y = scale * table[ids], zero where an id lies outside [0, V). The table
    [V, d] is an fp32 buffer, not a parameter, as ProjectedLinear's W is: it
    gets no gradient of its own. Given to a GrapeOptimizer it is updated
    privately; otherwise it stays as it is. The output requires grad, so that
    autograd reaches every layer after it."""

    def __init__(self, V: int, d: int, layer_id: int,
                 table: Optional[torch.Tensor] = None, scale: float = 1.0,
                 dtype: torch.dtype = torch.bfloat16, device="cuda"):
        super().__init__()
        if table is None:
            table = torch.randn(V, d, device=device) / math.sqrt(d)
        if tuple(table.shape) != (V, d):
            raise ValueError("table must be [V, d]")
        self.register_buffer("table", table.detach().to(torch.float32).contiguous())
        self.layer_id = int(layer_id)
        self.scale, self.dtype = float(scale), dtype
        self._grape = None  # the GrapeOptimizer driving this table, if any

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        ids = ids.contiguous()
        y = _b.dpg_embed(ids, self.table, scale=self.scale, dtype=self.dtype)
        if torch.is_grad_enabled():
            y.requires_grad_()
            if self._grape is not None:
                self._grape._capture_tokens(self, ids, y)
        return y


class _FirstDerivative(torch.autograd.Function):
    """A gradient as a function of what it was computed from, without a derivative
    of its own: the library has none, and a gradient without a graph would count as
    a constant in a second backward pass."""

    @staticmethod
    def forward(ctx, grad, *inputs):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the token losses have no second derivative")


def _gradients(grads, *inputs):
    # grad mode is on in a backward pass only when it builds a graph itself
    if torch.is_grad_enabled():
        return tuple(None if g is None else _FirstDerivative.apply(g, *inputs) for g in grads)
    return tuple(grads)


class _VocabLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, E, targets, scale):
        loss, lse = _b.dpg_vocab_loss(X, E, targets, scale=scale)
        ctx.save_for_backward(X, E, targets, lse)
        ctx.scale = scale
        return loss

    @staticmethod
    def backward(ctx, dloss):
        X, E, targets, lse = ctx.saved_tensors
        dX, dE = _b.dpg_vocab_loss_grad(X, E, targets, lse, dloss.contiguous(),
                                        scale=ctx.scale, need_dX=ctx.needs_input_grad[0],
                                        need_dE=ctx.needs_input_grad[1])
        return (*_gradients((dX, dE), X, E, dloss), None, None)


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, E, top_ids, top_logits, temperature, scale):
        loss, lse = _b.dpg_distill_loss(X, E, top_ids, top_logits, temperature=temperature,
                                        scale=scale)
        ctx.save_for_backward(X, E, top_ids, top_logits, lse)
        ctx.args = dict(temperature=temperature, scale=scale)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        X, E, top_ids, top_logits, lse = ctx.saved_tensors
        dX, dE = _b.dpg_distill_loss_grad(X, E, top_ids, top_logits, lse, dloss.contiguous(),
                                          need_dX=ctx.needs_input_grad[0],
                                          need_dE=ctx.needs_input_grad[1], **ctx.args)
        return (*_gradients((dX, dE), X, E, dloss), None, None, None, None)


def vocab_cross_entropy(X: torch.Tensor, E: torch.Tensor, targets: torch.Tensor,
                        scale: float = 1.0) -> torch.Tensor:
    """Per-row softmax cross entropy of X [..., d] against the table E [V, d]
    (same type) without an array of logits; differentiable once in X and E. Rows
    whose target lies outside [0, V) give 0. Returns fp32 of X's leading shape.
    E's gradient is an ordinary one: no call gives its norms per sample, so a table
    trained by it is outside a GrapeOptimizer's clip."""
    return _VocabLoss.apply(X.contiguous(), E.contiguous(), targets.contiguous(), scale)


def distill_cross_entropy(X: torch.Tensor, E: torch.Tensor, top_ids: torch.Tensor,
                          top_logits: torch.Tensor, temperature: float = 1.0,
                          scale: float = 1.0) -> torch.Tensor:
    """Per-row tau^2 KL of X [..., d] against the table E [V, d] from a teacher's
    top k logits (top_ids, top_logits [..., k]); differentiable once in X and E. The
    teacher's logits are data: they get no gradient, and ones that ask for one
    are refused (detach them)."""
    if torch.is_grad_enabled() and top_logits.requires_grad:
        raise ValueError("top_logits must not require grad: the teacher gets no gradient")
    return _DistillLoss.apply(X.contiguous(), E.contiguous(), top_ids.contiguous(),
                              top_logits.contiguous(), temperature, scale)
