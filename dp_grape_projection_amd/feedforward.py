"""The gated feed-forward block around the private update step, as a torch function and
as a module whose two linear layers can take part in the step of a GrapeOptimizer. All of
it runs in libdpg's kernels; this module only wires tensors to those calls.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch
from torch.autograd.forward_ad import unpack_dual

from . import binding as _b
from .streaming import ProjectedLinear


def _check_checkpoint(checkpoint):
    if checkpoint not in (None, "int8"):
        raise ValueError(f"checkpoint must be None or \"int8\", got {checkpoint!r}")


class _GatedBlock(torch.autograd.Function):
    """driver: None, or the (optimizer, up, down) that take the per-sample gradients of
    the block's layers when its backward pass runs."""

    @staticmethod
    def forward(ctx, X, W_in, W_out, act, checkpoint, driver):
        ctx.act, ctx.driver, ctx.int8 = act, driver, checkpoint == "int8"
        Y, Z = _b.dpg_gated(X, W_in, W_out, act=act, keep=ctx.int8)
        kept = [X]
        if ctx.int8:
            kept = [Z.codes, Z.exps]
            if driver is not None or ctx.needs_input_grad[1]:
                x8 = _b.dpg_pack_act(X)
                kept += [x8.codes, x8.exps]
        ctx.save_for_backward(W_in, W_out, *kept)
        return Y

    @staticmethod
    def backward(ctx, dY):
        # grad mode is on in a backward pass only when it builds a graph itself, in which
        # these gradients would count as constants
        if torch.is_grad_enabled():
            raise RuntimeError("the gated block has no second derivative (create_graph)")
        W_in, W_out, *kept = ctx.saved_tensors
        X, Z = kept[0].detach(), None
        if ctx.int8:
            d, f = (int(n) for n in reversed(W_out.shape))
            Z = _b.PackedActivations(kept[0], kept[1], f, W_in.dtype)
            X = _b.PackedActivations(kept[2], kept[3], d, W_in.dtype) if len(kept) > 2 else None
        dY = dY.contiguous()
        need_dX, *need_dW = ctx.needs_input_grad[:3]
        g = _b.dpg_gated_grad(dY, X, W_in, W_out, act=ctx.act, Z=Z, need_dX=need_dX,
                              need_dW=need_dW, need_layers=ctx.driver is not None)
        if ctx.driver is not None:
            optimizer, up, down = ctx.driver
            optimizer._project(up, X, g.dZ)
            optimizer._project(down, g.H, dY)
        return g.dX, g.dW_in, g.dW_out, None, None, None


def _gated_block(X, W_in, W_out, act, checkpoint, driver):
    X, W_in, W_out = X.contiguous(), W_in.contiguous(), W_out.contiguous()
    if torch.is_grad_enabled() and any(t.requires_grad for t in (X, W_in, W_out)):
        return _GatedBlock.apply(X, W_in, W_out, act, checkpoint, driver)
    # (the library's call would lose a tangent, which reads as a derivative of zero)
    if any(unpack_dual(t).tangent is not None for t in (X, W_in, W_out)):
        raise NotImplementedError("the gated block has no forward mode")
    return _b.dpg_gated(X, W_in, W_out, act=act)[0]


def gated_feed_forward(X: torch.Tensor, W_in: torch.Tensor, W_out: torch.Tensor,
                       act: str = "silu", checkpoint: Optional[str] = None) -> torch.Tensor:
    """(act(X W_gate) * (X W_up)) W_out of X [..., d], W_in = [W_gate | W_up] [d, 2 f] and
    W_out [f, d] in one type (bf16 or fp32); act "silu", "gelu" or "gelu_tanh".
    Differentiable once in all three, backwards; a backward pass that builds a graph of its
    own is refused, and so is forward mode. What is kept until then: with checkpoint None X
    alone, from which both projections are computed again; with "int8" both projections and
    (for W_in's gradient) X in 8 bits, whose gradients are those at the kept values."""
    _check_checkpoint(checkpoint)
    return _gated_block(X, W_in, W_out, act, checkpoint, None)


class GatedFeedForward(torch.nn.Module):
    """The gated block with its weights in two ProjectedLinear layers, `up` [d, 2 f] and
    `down` [f, d], fp32 buffers as theirs are. Given to a GrapeOptimizer (linears()) both
    are updated privately: the block's backward pass hands it their inputs and output
    gradients. x must then be [B, T, d] and require grad. The products run in x's type: a
    forward pass in bf16 casts both weights first (4 rows x 2048 x 8192 in a loop: 73 us, 25
    for gated_feed_forward of weights in bf16), and the copies live until the backward pass,
    beside what checkpoint keeps, which is as in gated_feed_forward."""

    def __init__(self, d: int, f: int, layer_ids: Sequence[int], act: str = "silu",
                 checkpoint: Optional[str] = None, W_in: Optional[torch.Tensor] = None,
                 W_out: Optional[torch.Tensor] = None, device="cuda"):
        super().__init__()
        _check_checkpoint(checkpoint)
        if act not in _b.ACTIVATIONS:
            raise ValueError(f"act must be one of {sorted(_b.ACTIVATIONS)}, got {act!r}")
        up_id, down_id = layer_ids
        self.up = ProjectedLinear(d, 2 * f, up_id, W=W_in, device=device)
        self.down = ProjectedLinear(f, d, down_id, W=W_out, device=device)
        self.act, self.checkpoint = act, checkpoint

    def linears(self):
        return [self.up, self.down]

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        driver = None
        optimizer = self.up._grape
        if optimizer is not self.down._grape:
            raise RuntimeError("one optimizer must drive both of the block's layers, or none")
        if optimizer is not None and torch.is_grad_enabled() and x.requires_grad:
            if x.dim() != 3:
                raise ValueError("x must be [B, T, d]")
            optimizer._begin_layer(x)
            driver = (optimizer, self.up, self.down)
        return _gated_block(x, self.up.W.to(x.dtype), self.down.W.to(x.dtype), self.act,
                            self.checkpoint, driver)
