"""The token operators inside the private step: a GrapeOptimizer with a token
embedding, and the example that runs all of them together.

The table's update is checked against the float64 reference on the ids and
gradients of the step, and the sample norms against the projected layers' own
norms plus the embedding's. Bars: fp32 1e-5, as in the other parity tests."""
import os
import sys

import numpy as np
import pytest

from _helpers import rel_err
from oracle import tokens as ot

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


@pytest.mark.parametrize("sigma", [0.0, 0.7])
def test_table_takes_part_in_the_private_step(sigma):
    import torch
    import dp_grape_projection_amd as dpg
    torch.manual_seed(1)
    V, d, B, T = 37, 24, 5, 11
    emb = dpg.TokenEmbedding(V, d, layer_id=9, scale=1.5, dtype=torch.float32)
    lin = dpg.ProjectedLinear(d, 16, layer_id=4)
    head = torch.randn(V, 16, device="cuda")
    opt = dpg.GrapeOptimizer([lin], r=8, clip_C=0.05, sigma=sigma, seed=3, lr=1e-2,
                             embeddings=[emb], table_lr=0.5)
    ids = torch.randint(-3, V, (B, T), device="cuda")
    ids[4] = -1                                  # a sample of padding only
    targets = torch.where(ids >= 0, (ids * 7 + 1) % V, -1)
    old = _host(emb.table)
    opt.zero_grad()
    loss = dpg.vocab_cross_entropy(lin(emb(ids)), head, targets)
    (loss / T).sum().backward()
    tok, dY = opt.tokens[9]
    dY = _host(dY)
    lin_sq = (_host(opt.G_hat[4]) ** 2).sum((1, 2))
    opt.step()
    torch.cuda.synchronize()
    ids_h = ids.cpu().numpy()
    norms = np.sqrt(lin_sq + ot.embed_norms_sq(ids_h, dY, V, 1.5))
    assert norms[4] == 0.0 and (norms[:4] > 0.05).any()
    assert rel_err(_host(opt.last_norms), norms) <= 1e-5
    s = np.minimum(1.0, 0.05 / np.where(norms > 0, norms, 1e-30))
    G = ot.embed_grad(ids_h, dY, V, 1.5, s)
    if sigma:
        G = G + sigma * 0.05 * _host(dpg.dpg_philox_normals(3, 9, 1, 1, 0, V * d)).reshape(V, d)
    # the stored table adds one rounding of its own values
    got = (_host(emb.table) - old) * (-B / 0.5)
    half = np.spacing(np.abs(old).astype(np.float32)).astype(np.float64) * (B / 0.5)
    assert (np.abs(got - G) <= 1e-5 * np.abs(G).max() + half).all()


def test_losses_through_autograd():
    import torch
    import dp_grape_projection_amd as dpg
    torch.manual_seed(2)
    X = torch.randn(3, 7, 24, device="cuda", requires_grad=True)
    E = torch.randn(91, 24, device="cuda", requires_grad=True)
    y = torch.randint(-5, 91, (3, 7), device="cuda")
    w = torch.rand(3, 7, device="cuda")
    (dpg.vocab_cross_entropy(X, E, y, scale=0.7) * w).sum().backward()
    yh = y.cpu().numpy()
    _, _, dX, dE = ot.target_loss(_host(X.detach()), _host(E.detach()), yh, (yh >= 0) * 1.0,
                                  0.7, 1.0, _host(w))
    assert rel_err(_host(X.grad), dX) <= 1e-5
    assert rel_err(_host(E.grad), dE) <= 1e-5
    top = torch.stack([y, (y + 13) % 91], -1)
    t = torch.randn(3, 7, 2, device="cuda")
    frozen = E.detach()
    X.grad = None
    (dpg.distill_cross_entropy(X, frozen, top, t, temperature=3.0) * w).sum().backward()
    q = ot.teacher_weights(top.cpu().numpy(), t.cpu().numpy(), 91, 3.0)
    _, _, dX, _ = ot.target_loss(_host(X.detach()), _host(frozen), top.cpu().numpy(), q, 1.0, 3.0,
                                 _host(w))
    assert rel_err(_host(X.grad), dX) <= 1e-5


def test_example_learns():
    import private_lm
    losses = private_lm.train(steps=40)
    assert np.isfinite(losses).all()
    assert np.mean(losses[-5:]) < np.mean(losses[:5]) - 0.3, losses


def test_a_table_without_gradient_is_reported():
    import torch
    import dp_grape_projection_amd as dpg
    emb = dpg.TokenEmbedding(5, 8, layer_id=0, dtype=torch.float32)
    opt = dpg.GrapeOptimizer([dpg.ProjectedLinear(8, 8, layer_id=1)], r=4, clip_C=1.0, sigma=0.0,
                             seed=0, lr=1e-3, embeddings=[emb])
    with pytest.raises(RuntimeError):
        emb(torch.zeros((1, 2), dtype=torch.int64, device="cuda"))   # before zero_grad
    opt.zero_grad()
    with pytest.raises(RuntimeError):
        opt.step()
    with pytest.raises(ValueError):
        dpg.GrapeOptimizer([dpg.ProjectedLinear(8, 8, layer_id=0)], r=4, clip_C=1.0, sigma=0.0,
                           seed=0, lr=1e-3, embeddings=[emb])
