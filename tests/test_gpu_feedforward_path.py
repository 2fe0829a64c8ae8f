"""The feed-forward operators as a program uses them: the block under autograd, its layers
and 8-bit inputs in a GrapeOptimizer's private step, and the example that trains with
them.

Bars: fp32 1e-5 (products of exact parts, sums in fp32), bf16 2e-2 for projected
gradients (P and A P^T rounded), as in the other tests of the step."""
import os
import sys

import numpy as np
import pytest

import oracle
from _helpers import TOL, rel_err
from oracle import feedforward as of

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _host(t):
    return t.double().cpu().numpy()


def _leaves(d, f, lead=(3, 7), dtype=None, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = ((*lead, d), (d, 2 * f), (f, d))
    return [torch.randn(s, generator=g, device="cuda").to(dtype or torch.float32).requires_grad_()
            for s in shapes]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_autograd(act, checkpoint):
    import torch
    import dp_grape_projection_amd as dpg
    X, W_in, W_out = _leaves(24, 40)
    w = torch.randn(3, 7, 24, device="cuda")
    Y = dpg.gated_feed_forward(X, W_in, W_out, act=act, checkpoint=checkpoint)
    grads = torch.autograd.grad((Y * w).sum(), [X, W_in, W_out])
    x, wi, wo, dy = (_host(t.detach()).reshape(-1, t.shape[-1]) for t in (X, W_in, W_out, w))
    want, G, U = of.gated(x, wi, wo, act)
    assert rel_err(_host(Y.detach()).reshape(-1, 24), want) <= 1e-5
    if checkpoint:
        _, Z = dpg.dpg_gated(X.detach(), W_in.detach(), W_out.detach(), act=act, keep=True)
        z = _host(dpg.dpg_unpack_act(Z)).reshape(-1, 2, 40)
        G, U = z[:, 0], z[:, 1]
        x = _host(dpg.dpg_unpack_act(dpg.dpg_pack_act(X.detach()))).reshape(-1, 24)
    for got, ref in zip(grads, of.gated_grad(dy, x, G, U, wi, wo, act)):
        assert rel_err(_host(got).reshape(ref.shape), ref) <= 1e-5


def test_gradient_against_differences():
    """fp32: a difference over 2 h of a sum of values near 1 is off by at most 2^-23
    |sum| / h and h^2 third derivatives; h = 2^-6 and directions of all elements."""
    import torch
    import dp_grape_projection_amd as dpg
    X, W_in, W_out = (t.detach() / 4 for t in _leaves(16, 24, lead=(5,), seed=4))
    for t in (X, W_in, W_out):
        t.requires_grad_()
    w = torch.randn(5, 16, device="cuda")
    Y = dpg.gated_feed_forward(X, W_in, W_out)
    grads = torch.autograd.grad((Y * w).sum(), [X, W_in, W_out])
    h = 2.0 ** -6
    for i in range(3):
        v = torch.randn_like(grads[i])
        side = []
        for s in (h, -h):
            args = [t.detach().clone() for t in (X, W_in, W_out)]
            args[i] += s * v
            side.append(float((dpg.gated_feed_forward(*args).double() * w).sum()))
        got, want = (side[0] - side[1]) / (2 * h), float((grads[i].double() * v).sum())
        scale = float((grads[i].abs() * v.abs()).sum())
        assert abs(got - want) <= 1e-2 * scale


def test_needs_and_refusals():
    import torch
    import dp_grape_projection_amd as dpg
    for checkpoint in (None, "int8"):
        X, W_in, W_out = _leaves(32, 64, dtype=torch.bfloat16)
        full = torch.autograd.grad(
            dpg.gated_feed_forward(X, W_in, W_out, checkpoint=checkpoint).float().sum(), [X, W_in, W_out])
        for i, on in enumerate(((1, 0, 0), (0, 1, 0), (0, 0, 1))):
            args = [t.detach().requires_grad_(bool(o)) for t, o in zip((X, W_in, W_out), on)]
            dpg.gated_feed_forward(*args, checkpoint=checkpoint).float().sum().backward()
            assert [a.grad is not None for a in args] == [bool(o) for o in on]
            assert torch.equal(args[i].grad, full[i])
        # a batch that is a view of another order, and weights that are
        Xt = X.detach().transpose(0, 1).contiguous().transpose(0, 1).requires_grad_()
        Y = dpg.gated_feed_forward(Xt, W_in.detach().t().contiguous().t(), W_out, checkpoint=checkpoint)
        dX, = torch.autograd.grad(Y.float().sum(), [Xt])
        assert torch.equal(dX, full[0])
        # twice through one graph; a graph of the gradients is refused
        Y = dpg.gated_feed_forward(X, W_in, W_out, checkpoint=checkpoint)
        for _ in range(2):
            again = torch.autograd.grad(Y.float().sum(), [X, W_in, W_out], retain_graph=True)
            assert all(torch.equal(a, b) for a, b in zip(again, full))
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(Y.float().sum(), [X], create_graph=True)
        with torch.no_grad():
            Y0 = dpg.gated_feed_forward(X, W_in, W_out, checkpoint=checkpoint)
        assert torch.equal(Y0, Y) and not Y0.requires_grad
    with pytest.raises(TypeError):
        dpg.gated_feed_forward(X.float(), W_in, W_out)


def test_8_bits_are_what_stays():
    """Between the passes of a block with checkpoint "int8" its graph holds 1.03 bytes for
    every element of X and of both projections, and no projection in 16 bits."""
    import torch
    import dp_grape_projection_amd as dpg
    N, d, f = 4096, 512, 2048
    W_in, W_out = (t.requires_grad_() for t in (
        torch.randn(d, 2 * f, device="cuda", dtype=torch.bfloat16),
        torch.randn(f, d, device="cuda", dtype=torch.bfloat16)))
    held = {}
    for checkpoint in (None, "int8"):
        x = torch.randn(N, d, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        Y = dpg.gated_feed_forward(x, W_in, W_out, checkpoint=checkpoint)
        del x
        held[checkpoint] = torch.cuda.memory_allocated() - before - Y.numel() * 2
        Y.float().sum().backward()
        del Y
    packed = lambda n: n + n // 32  # noqa: E731
    assert held["int8"] <= packed(N * 2 * f) + packed(N * d) - N * d * 2 + (1 << 16)
    assert held[None] <= 1 << 16


def _check_private(opt, layers, old, r, seed, dtype, t=1):
    """G_priv and the norms against the formula on what the layers were given."""
    import dp_grape_projection_amd as dpg
    norms_sq, hats = 0.0, []
    for layer in layers:
        A, dY = opt.inputs[layer.layer_id]
        if isinstance(A, dpg.PackedActivations):
            A = dpg.dpg_unpack_act(A)
        P = oracle.projection_matrix(seed, layer.layer_id, t, r, layer.d_in)
        hat = np.stack([P @ (_host(A[i]).T @ _host(dY[i])) for i in range(A.shape[0])])
        norms_sq = norms_sq + np.sum(hat ** 2, axis=(1, 2))
        hats.append(hat)
    n = np.sqrt(norms_sq)
    assert rel_err(_host(opt.last_norms), n) <= TOL[dtype]
    s = np.minimum(1.0, opt.clip_C / n)
    for hat, got in zip(hats, opt.last_G_priv):
        assert rel_err(_host(got), np.einsum("i,ijk->jk", s, hat) / len(n)) <= TOL[dtype]
    for layer, w in zip(layers, old):
        assert np.abs(_host(layer.W) - w).max() > 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_block_in_the_private_step(checkpoint, dtype):
    """A block between two projected layers: its layers get the gradients that the same
    weights get as layers of their own with torch's activation between them."""
    import torch
    import dp_grape_projection_amd as dpg
    torch.manual_seed(5)
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    B, T, d, f, r = 4, 10, 24, 40, 8
    first, block = dpg.ProjectedLinear(d, d, 11), dpg.GatedFeedForward(
        d, f, (3, 7), act="gelu", checkpoint=checkpoint)
    layers = [first, *block.linears()]
    opt = dpg.GrapeOptimizer(layers, r=r, clip_C=0.01, sigma=0.0, seed=9, lr=1e-2,
                             keep_inputs=True, checkpoint=checkpoint)
    x = torch.randn(B, T, d, device="cuda", dtype=dt).requires_grad_()
    w = torch.randn(B, T, d, device="cuda", dtype=dt) / T
    old = [_host(l.W) for l in layers]
    opt.zero_grad()
    y = block(first(x))
    (y * w).float().sum().backward()
    assert isinstance(opt.inputs[3][0], dpg.PackedActivations) == (checkpoint == "int8")
    dZ, H = opt.inputs[3][1], opt.inputs[7][0]
    opt.step()
    torch.cuda.synchronize()
    _check_private(opt, layers, old, r, 9, dtype)
    if checkpoint is None and dtype == "fp32":
        # the same gradients by torch's own layers
        h = (x @ torch.from_numpy(old[0]).cuda().float()).detach()
        z = (h.double() @ torch.from_numpy(old[1]).cuda()).requires_grad_()
        hidden = torch.nn.functional.gelu(z[..., :f]) * z[..., f:]
        (dz,) = torch.autograd.grad(hidden, z, w.double() @ torch.from_numpy(old[2]).cuda().t())
        assert rel_err(_host(dZ), _host(dz)) <= 1e-5
        assert rel_err(_host(H), _host(hidden.detach())) <= 1e-5


def test_block_misused():
    import torch
    import dp_grape_projection_amd as dpg
    block = dpg.GatedFeedForward(8, 16, (0, 1))
    opt = dpg.GrapeOptimizer(block.linears(), r=4, clip_C=1.0, sigma=0.0, seed=0, lr=0.1)
    x = torch.randn(2, 3, 8, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="zero_grad"):
        block(x)
    opt.zero_grad()
    with pytest.raises(ValueError, match="B, T, d"):
        block(x[0])
    block(x).sum().backward()
    with pytest.raises(RuntimeError, match="twice"):
        block(x).sum().backward()
    opt.step()
    with torch.no_grad():
        assert tuple(block(x[0]).shape) == (3, 8)


def test_inputs_in_8_bits_in_the_private_step():
    """Plain layers whose inputs the optimizer keeps in 8 bits, over two steps."""
    import torch
    import dp_grape_projection_amd as dpg
    torch.manual_seed(6)
    layers = [dpg.ProjectedLinear(40, 72, 5), dpg.ProjectedLinear(72, 16, 2)]
    opt = dpg.GrapeOptimizer(layers, r=16, clip_C=0.02, sigma=0.0, seed=4, lr=1e-2,
                             keep_inputs=True, checkpoint="int8")
    for t in (1, 2):
        x = torch.randn(3, 12, 40, device="cuda").requires_grad_()
        w = torch.randn(3, 12, 16, device="cuda") / 12
        old = [_host(l.W) for l in layers]
        opt.zero_grad()
        (layers[1](torch.tanh(layers[0](x))) * w).sum().backward()
        opt.step()
        torch.cuda.synchronize()
        for i in (5, 2):
            assert isinstance(opt.inputs[i][0], dpg.PackedActivations)
        _check_private(opt, layers, old, 16, 4, "fp32", t)
    want = dpg.dpg_pack_act(x.detach())
    assert torch.equal(opt.inputs[5][0].codes, want.codes)


def test_example_runs_with_gated_blocks():
    import math
    import torch
    import private_lm
    keep = []
    losses = private_lm.train(steps=2, V=128, d=32, B=8, T=16, gated=True, keep=keep)
    opt, model = keep
    assert len(losses) == 2 and all(math.isfinite(v) for v in losses)
    assert len(opt.layers) == 4 and all(len(b.linears()) == 2 for b in model.blocks)
    assert all(torch.isfinite(l.W).all() for l in opt.layers)
