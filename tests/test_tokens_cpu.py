"""The modules and functions around the token operators on the CPU: the library's
calls are replaced by their formulas in torch, so that what tokens.py and
streaming.py do with them can be tested without a GPU."""
import math

import pytest
import torch

import dp_grape_projection_amd as dpg
from dp_grape_projection_amd import binding


def _vocab(X, E, targets, scale):
    z = scale * X.flatten(0, -2) @ E.t()
    y = targets.flatten()
    on = (y >= 0) & (y < E.shape[0])
    at = torch.where(on, y, 0)[:, None]
    return z, on, torch.zeros_like(z).scatter_(1, at, 1.0) * on[:, None]


def _losses(z, on, q, shape):
    lse = torch.logsumexp(z, 1) * on
    return ((lse - (z * q).sum(1)) * on).view(shape), lse.view(shape)


def _grads(z, on, q, X, E, dloss, factor, need_dX, need_dE):
    D = (torch.softmax(z, 1) * on[:, None] - q) * (factor * dloss.flatten()[:, None])
    return ((D @ E).view(X.shape) if need_dX else None,
            D.t() @ X.flatten(0, -2) if need_dE else None)


@pytest.fixture
def formulas(monkeypatch):
    """dpg_vocab_loss and dpg_distill_loss with their gradients, as formulas. Like the
    library's, their outputs carry no graph."""
    @torch.no_grad()
    def vocab(X, E, targets, scale=1.0):
        return _losses(*_vocab(X, E, targets, scale), X.shape[:-1])

    @torch.no_grad()
    def vocab_grad(X, E, targets, lse, dloss, scale=1.0, need_dX=True, need_dE=True):
        return _grads(*_vocab(X, E, targets, scale), X, E, dloss, scale, need_dX, need_dE)

    def teacher(X, E, top_ids, top_logits, tau, scale):
        z = scale / tau * X.flatten(0, -2) @ E.t()
        q = torch.softmax(top_logits.flatten(0, -2) / tau, 1)
        q = torch.zeros_like(z).scatter_add_(1, top_ids.flatten(0, -2), q)
        return z, torch.ones(z.shape[0], dtype=torch.bool), q

    @torch.no_grad()
    def distill(X, E, top_ids, top_logits, temperature=1.0, scale=1.0):
        return _losses(*teacher(X, E, top_ids, top_logits, temperature, scale), X.shape[:-1])

    @torch.no_grad()
    def distill_grad(X, E, top_ids, top_logits, lse, dloss, temperature=1.0, scale=1.0,
                     need_dX=True, need_dE=True):
        return _grads(*teacher(X, E, top_ids, top_logits, temperature, scale), X, E, dloss,
                      scale * temperature, need_dX, need_dE)

    for name, fn in (("dpg_vocab_loss", vocab), ("dpg_vocab_loss_grad", vocab_grad),
                     ("dpg_distill_loss", distill), ("dpg_distill_loss_grad", distill_grad)):
        monkeypatch.setattr(binding, name, fn)


def _loss_inputs():
    g = torch.Generator().manual_seed(4)
    X = torch.randn(2, 3, 8, generator=g, requires_grad=True)
    E = torch.randn(11, 8, generator=g, requires_grad=True)
    y = torch.randint(0, 11, (2, 3), generator=g)
    top = torch.stack([y, (y + 3) % 11], -1)
    return X, E, y, top, torch.randn(2, 3, 2, generator=g)


def _loss(which, X, E, y, top, t):
    if which == "vocab":
        return dpg.vocab_cross_entropy(X, E, y, scale=0.7)
    return dpg.distill_cross_entropy(X, E, top, t, temperature=1.5)


@pytest.mark.parametrize("which", ["vocab", "distill"])
@pytest.mark.parametrize("weighted", [False, True])
def test_a_second_derivative_is_refused(formulas, which, weighted):
    """A penalty on the gradient must not lose its part of the result silently,
    whether or not what arrives at the loss's backward has a graph of its own."""
    X, E, y, top, t = _loss_inputs()
    w = torch.ones(2, 3, requires_grad=weighted)
    total = (_loss(which, X, E, y, top, t) * w).sum()
    dX, dE = torch.autograd.grad(total, (X, E), create_graph=True)
    for part in (dX, dE):
        with pytest.raises(RuntimeError, match="second derivative"):
            (part.square().sum() + X.sum() + E.sum()).backward(retain_graph=True)


@pytest.mark.parametrize("which", ["vocab", "distill"])
def test_a_first_derivative_that_keeps_its_graph(formulas, which):
    """create_graph alone changes no value."""
    X, E, y, top, t = _loss_inputs()
    want = torch.autograd.grad(_loss(which, X, E, y, top, t).sum(), (X, E))
    got = torch.autograd.grad(_loss(which, X, E, y, top, t).sum(), (X, E), create_graph=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    frozen = E.detach()
    dX, = torch.autograd.grad(_loss(which, X, frozen, y, top, t).sum(), X, create_graph=True)
    assert torch.equal(dX, want[0])


def test_a_teacher_that_wants_a_gradient_is_refused(formulas):
    X, E, y, top, t = _loss_inputs()
    t.requires_grad_()
    with pytest.raises(ValueError, match="top_logits"):
        dpg.distill_cross_entropy(X, E, top, t)
    with torch.no_grad():                        # nothing is lost without a graph
        dpg.distill_cross_entropy(X, E, top, t)
    dpg.distill_cross_entropy(X, E, top, t.detach()).sum().backward()
    assert X.grad is not None and t.grad is None


# ------------------------------------------- the table in the private step --

V, D_IN, D_OUT = 9, 6, 4


def _table_sum(ids, dY, V, scale, s):
    G = torch.zeros(V, dY.shape[-1])
    for b, row in enumerate(ids.tolist()):
        for t, v in enumerate(row):
            if 0 <= v < V:
                G[v] += scale * float(s[b]) * dY[b, t]
    return G


@pytest.fixture
def private(monkeypatch):
    """A table and a projected layer under a GrapeOptimizer, on the CPU; `calls`
    lists the library's calls in order, `fail` names one that raises."""
    class Setup:
        calls, fail = [], None

    def step_call(fn):
        def wrapper(*args, **kw):
            Setup.calls.append(fn.__name__)
            if Setup.fail == fn.__name__:
                raise RuntimeError(fn.__name__)
            with torch.no_grad():
                return fn(*args, **kw)
        monkeypatch.setattr(binding, fn.__name__, wrapper)

    @step_call
    def dpg_embed(ids, E, scale=1.0, dtype=None):
        if not ids.is_contiguous():
            raise ValueError("ids must be contiguous")
        ok = (ids >= 0) & (ids < E.shape[0])
        return (scale * E[torch.where(ok, ids, 0)] * ok[..., None]).to(dtype or E.dtype)

    @step_call
    def dpg_embed_norms(ids, dY, V, norm_sq, scale=1.0):
        if not ids.is_contiguous():
            raise ValueError("ids must be contiguous")
        for b in range(ids.shape[0]):
            norm_sq[b] += _table_sum(ids[b:b + 1], dY[b:b + 1], V, scale, [1.0]).square().sum()

    @step_call
    def dpg_embed_grad(ids, dY, V, scale=1.0, sample_scales=None):
        return _table_sum(ids, dY, V, scale, sample_scales)

    @step_call
    def dpg_philox_normals(seed, layer_id, step_word, tag, start, n, device=None):
        return torch.randn(n, generator=torch.Generator().manual_seed(seed))

    @step_call
    def dpg_project_layer(A, dY, r, seed, proj_step, layer_id, norm_sq, G_hat=None):
        G = torch.einsum("btk,bto->bko", A, dY)[:, :r].contiguous()
        norm_sq += G.square().sum((1, 2))
        return G

    @step_call
    def dpg_clip_sum_noise(G_hat, r, C, sigma, seed, step, norm_sq, layer_ids=None):
        norms = norm_sq.sqrt()
        s = torch.clamp(C / norms, max=1.0)[:, None, None]
        return [(s * G).sum(0) for G in G_hat], norms

    @step_call
    def dpg_adam_backproject(G, W, m, v, r, lr, *args, **kw):
        for w, g in zip(W, G):
            w[:r] -= lr * g

    def build(sigma=0.0, **kw):
        torch.manual_seed(3)
        Setup.emb = dpg.TokenEmbedding(V, D_IN, layer_id=1, scale=1.5, dtype=torch.float32,
                                       device="cpu")
        Setup.lin = dpg.ProjectedLinear(D_IN, D_OUT, layer_id=2, device="cpu")
        Setup.opt = dpg.GrapeOptimizer([Setup.lin], r=3, clip_C=0.3, sigma=sigma, seed=5, lr=0.1,
                                       embeddings=[Setup.emb], table_lr=0.5, **kw)
        Setup.calls.clear()
        return Setup
    Setup.build = staticmethod(build)
    return Setup


def _ids():
    return torch.tensor([[0, 4, 4, -1], [8, 0, 2, 2], [7, 7, 7, 7]])


def _step(s, ids, between=()):
    """One step; between: what happens after the forward pass, the backward pass."""
    s.opt.zero_grad()
    y = s.emb(ids)
    out = s.lin(y)
    for fn in between[:1]:
        fn(y)
    (out * torch.arange(1.0, 13.0).view(3, 4, 1)).sum().backward()
    for fn in between[1:]:
        fn(y)
    s.opt.step()
    return s.emb.table.clone()


@pytest.mark.parametrize("when", ["after the forward pass", "after the backward pass"])
def test_a_refilled_id_buffer_does_not_reach_the_step(private, when):
    """Norms, clip factors and the gradient belong to the ids of the lookup."""
    want = _step(private.build(), _ids())
    ids = _ids()

    def refill(y):
        ids.copy_((ids + 3) % V)
    keep = lambda y: None
    got = _step(private.build(), ids, (refill, keep) if "forward" in when else (keep, refill))
    assert torch.equal(got, want)


def test_a_changed_gradient_is_reported(private):
    """The table's gradient must be the one whose norms were taken."""
    s = private.build()
    old = s.emb.table.clone()
    with pytest.raises(RuntimeError, match="changed"):
        _step(s, _ids(), (lambda y: None, lambda y: y.grad.mul_(100.0)))
    assert torch.equal(s.emb.table, old)


@pytest.mark.parametrize("fail", ["dpg_embed_grad", "dpg_philox_normals", "dpg_clip_sum_noise",
                                  "dpg_adam_backproject"])
def test_a_step_that_fails_changes_nothing(private, fail):
    """What can fail comes before the first write to a weight or a table."""
    s = private.build(sigma=0.5)
    table, W = s.emb.table.clone(), s.lin.W.clone()
    s.fail = fail
    with pytest.raises(RuntimeError, match=fail):
        _step(s, _ids())
    assert torch.equal(s.emb.table, table) and torch.equal(s.lin.W, W)
    s.fail = None
    s.opt.step()                                 # and can be taken again
    assert not torch.equal(s.emb.table, table) and not torch.equal(s.lin.W, W)
    got, got_W = s.emb.table.clone(), s.lin.W.clone()
    other = private.build(sigma=0.5)
    assert torch.equal(_step(other, _ids()), got) and torch.equal(other.lin.W, got_W)


def test_a_table_past_the_noise_stream_is_refused():
    """The noise of one layer and step has fewer than 2^32 entries."""
    emb = dpg.TokenEmbedding(2 ** 21, 2 ** 11, layer_id=1, device="meta",
                             table=torch.empty((2 ** 21, 2 ** 11), device="meta"))
    lin = dpg.ProjectedLinear(D_IN, D_OUT, layer_id=2, device="cpu")
    args = dict(r=3, clip_C=1.0, seed=5, lr=0.1, embeddings=[emb])
    with pytest.raises(ValueError, match="2\\^32"):
        dpg.GrapeOptimizer([lin], sigma=0.5, **args)
    dpg.GrapeOptimizer([lin], sigma=0.0, **args)


def test_ids_of_any_strides(private):
    """A next-token split, seq[:, :-1], and a batch laid out the other way round."""
    want = _step(private.build(), _ids())
    seq = torch.cat([_ids(), _ids()[:, :1]], 1)
    assert torch.equal(_step(private.build(), seq[:, :-1]), want)
    assert torch.equal(_step(private.build(), _ids().t().contiguous().t()), want)
