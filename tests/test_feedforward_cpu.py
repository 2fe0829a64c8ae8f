"""What the gated block's torch function does around the library's calls, with those
calls replaced by elementary torch on the CPU."""
import numpy as np
import pytest
import torch

import dp_grape_projection_amd as dpg
from dp_grape_projection_amd import feedforward as ff
from oracle import feedforward as of


@pytest.fixture
def calls(monkeypatch):
    """The forward call in plain torch; the `keep` of every call."""
    kept = []

    def gated(X, W_in, W_out, act="silu", keep=False):
        kept.append(keep)
        g, u = (X @ W_in).chunk(2, dim=-1)
        Z = None
        if keep:
            lead, f = X.shape[:-1], int(W_out.shape[0])
            Z = dpg.PackedActivations(torch.zeros(*lead, 2, -(-f // 32) * 32, dtype=torch.int8),
                                      torch.zeros(*lead, 2, -(-f // 32), dtype=torch.uint8), f, X.dtype)
        return (torch.nn.functional.silu(g) * u) @ W_out, Z

    def pack(X):
        blocks = -(-int(X.shape[-1]) // 32)
        return dpg.PackedActivations(torch.zeros(*X.shape[:-1], 32 * blocks, dtype=torch.int8),
                                     torch.zeros(*X.shape[:-1], blocks, dtype=torch.uint8),
                                     int(X.shape[-1]), X.dtype)

    monkeypatch.setattr(ff._b, "dpg_gated", gated)
    monkeypatch.setattr(ff._b, "dpg_pack_act", pack)
    return kept


def _args(*requires_grad):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, generator=g).requires_grad_(bool(r))
            for s, r in zip(((2, 3, 4), (4, 12), (6, 4)), requires_grad)]


@pytest.mark.parametrize("checkpoint", [None, "int8"])
@pytest.mark.parametrize("wanted", [(0, 0, 0), (1, 1, 1)])
@pytest.mark.parametrize("grad_mode", [True, False])
def test_forward_mode_is_refused(calls, checkpoint, wanted, grad_mode):
    """A tangent that the block cannot carry on is an error, never a derivative of zero:
    with frozen weights, without a backward graph, in each of the inputs."""
    import torch.autograd.forward_ad as fwd
    for i in range(3):
        args = _args(*wanted)
        with fwd.dual_level(), torch.set_grad_enabled(grad_mode):
            args[i] = fwd.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(NotImplementedError):
                dpg.gated_feed_forward(*args, checkpoint=checkpoint)


def test_forward_mode_is_refused_by_the_module(calls):
    import torch.autograd.forward_ad as fwd
    block = dpg.GatedFeedForward(4, 6, (0, 1), device="cpu")
    x = _args(0, 0, 0)[0]
    with fwd.dual_level():
        with pytest.raises(NotImplementedError):
            block(fwd.make_dual(x, torch.ones_like(x)))
    assert not block(x).requires_grad


@pytest.mark.parametrize("wanted", [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1)])
def test_8_bits_are_written_only_for_a_backward_pass(calls, wanted):
    ff_args = _args(*wanted)
    with torch.no_grad():
        y0 = dpg.gated_feed_forward(*ff_args, checkpoint="int8")
    with torch.inference_mode():
        dpg.gated_feed_forward(*ff_args, checkpoint="int8")
    assert calls == [False, False] and not y0.requires_grad
    if not any(wanted):
        y = dpg.gated_feed_forward(*ff_args, checkpoint="int8")
        assert calls[-1] is False and not y.requires_grad
        assert torch.equal(y, y0)


def test_function_transforms_are_refused(calls):
    args = _args(0, 0, 0)
    tangents = [torch.ones_like(t) for t in args]
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(dpg.gated_feed_forward, tuple(args), tuple(tangents))
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.grad(lambda x: dpg.gated_feed_forward(x, *args[1:]).sum())(args[0])


def test_how_far_8_bits_are_off():
    """By 2^-7 of a block's largest magnitude or by 2^-127, whichever is more; either bound
    is met within a few percent, the second where the first would promise more."""
    r = np.random.default_rng(2)
    x = (r.uniform(-1, 1, (4000, 32)) * 2.0 ** r.integers(-140, 120, (4000, 1))).astype(np.float32)
    off = np.abs(of.unpack8(*of.pack8(x), 32) - x.astype(np.float64)).max(1)
    top = np.abs(x.astype(np.float64)).max(1)
    assert (off <= np.maximum(2.0 ** -7 * top, 2.0 ** -127)).all()
    large, small = top >= 2.0 ** -120, (top > 2.0 ** -127) & (top < 2.0 ** -121)
    assert (off[large] / top[large]).max() > 0.95 * 2.0 ** -7
    assert (off[small] / top[small]).max() > 2.0 ** -2 and off[small].max() > 0.95 * 2.0 ** -127
