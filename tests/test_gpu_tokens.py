"""GPU parity of the token operators (dpg_embed, dpg_embed_norms,
dpg_embed_grad, dpg_vocab_loss, dpg_distill_loss and their gradients) against
the float64 reference oracle.tokens, at small and ragged sizes, with
positions that take no part and poisoned data behind them.

Tolerances, per piece (tests/_helpers.rel_err). An fp32 output of sums of up
to a few thousand fp32 products: 1e-5, the fp32 bar of the other tests. A bf16
output is one rounding, relative 2^-9 at most; the losses' gradients carry a
second one of the same size (D in bf16 between the two products), and a piece
may hold less than its row's share of the norm: 2^-7. Losses and lse are sums
of logits of size a few units, taken absolutely: 2e-5 max(1, |lse|), twice the
fp32 bar since two terms of that size are subtracted."""
import math

import numpy as np
import pytest

from _helpers import rel_err
from oracle import tokens as ot

pytestmark = pytest.mark.gpu

TOL = {"fp32": 1e-5, "bf16": 2.0 ** -7}


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _dev(a, dtype=None, offset=0):
    """A contiguous device copy; offset elements off an aligned start."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}.get(dtype, t.dtype)
    flat = torch.empty(t.numel() + offset, dtype=dt, device="cuda")
    out = flat[offset:].view(t.shape)
    out.copy_(t)
    return out


def _host(t):
    return t.double().cpu().numpy()


def _round(a, dtype):
    """The values a tensor of `dtype` holds after rounding `a`."""
    import torch
    t = torch.from_numpy(np.asarray(a, np.float32))
    return (t.bfloat16() if dtype == "bf16" else t).double().numpy()


# -------------------------------------------------------------- embedding --

# B, T, d, V
EMBED = [
    (1, 1, 8, 1), (3, 7, 5, 13), (2, 300, 64, 50), (4, 33, 1002, 777), (1, 2100, 24, 3),
    (2, 5, 16, 1100), (64, 1, 2048, 5000), (5, 129, 40, 4099), (2, 1030, 136, 40),
]
TYPES = [("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")]   # table, activations


def _embed_case(B, T, d, V, seed):
    r = np.random.default_rng([B, T, d, V, seed])
    # frequent low ids, some positions out of the vocabulary on either side
    ids = np.minimum((V ** r.random((B, T))).astype(np.int64) - 1, V - 1)
    off = r.random((B, T)) < 0.15
    ids[off] = r.choice([-1, -7, V, V + 1, 2 ** 40, -2 ** 40], off.sum())
    if B > 1:
        ids[B - 1] = -1                   # a sample of padding only
    E = r.standard_normal((V, d))
    dY = r.standard_normal((B, T, d))
    s = (0.1 + r.random(B)).astype(np.float32)
    return ids, E, dY, s


@pytest.mark.parametrize("table,act", TYPES)
@pytest.mark.parametrize("B,T,d,V", EMBED)
def test_embed(B, T, d, V, table, act):
    import torch
    import dp_grape_projection_amd as dpg
    ids, E, _, _ = _embed_case(B, T, d, V, 1)
    E = _round(E, table)
    for offset in (0, 1):
        Y = dpg.dpg_embed(_dev(ids), _dev(E, table, offset), scale=1.7,
                          dtype=torch.bfloat16 if act == "bf16" else None)
        # one fp32 product (scale as fp32), rounded once
        want = (ot.embed(ids, E).astype(np.float32) * np.float32(1.7))
        np.testing.assert_array_equal(_host(Y), _round(want, act))


@pytest.mark.parametrize("table,act", TYPES)
@pytest.mark.parametrize("B,T,d,V", EMBED)
def test_embed_norms_and_grad(B, T, d, V, table, act):
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[embed] B={B} T={T} d={d} V={V} {table} {act}", flush=True)
    ids, _, dY, s = _embed_case(B, T, d, V, 2)
    dY = _round(dY, act)
    masked = (ids < 0) | (ids >= V)
    poisoned = dY.copy()
    poisoned[masked] = np.nan             # never read
    td = torch.bfloat16 if table == "bf16" else torch.float32
    base = np.linspace(0.5, 2.0, B)
    want_n = ot.embed_norms_sq(ids, dY, V, 1.3)
    want_g = ot.embed_grad(ids, dY, V, 1.3, s)
    old = _round(np.random.default_rng(3).standard_normal((V, d)), table)
    for offset in (0, 1):
        x = _dev(poisoned, act, offset)
        n2 = dpg.dpg_embed_norms(_dev(ids), x, V, _dev(base, "fp32"), scale=1.3)
        assert rel_err(_host(n2), base.astype(np.float32) + want_n) <= TOL["fp32"]
        dE = dpg.dpg_embed_grad(_dev(ids), x, V, 1.3, _dev(s), td,
                                dE=_dev(np.full((V, d), np.nan), table, offset))
        assert rel_err(_host(dE), want_g) <= TOL[table]
        again = dpg.dpg_embed_grad(_dev(ids), x, V, 1.3, _dev(s), td)
        assert torch.equal(dE, again)
        plain = dpg.dpg_embed_grad(_dev(ids), x, V, table_dtype=td)
        assert rel_err(_host(plain), ot.embed_grad(ids, dY, V)) <= TOL[table]
        acc = dpg.dpg_embed_grad(_dev(ids), x, V, 1.3, _dev(s), dE=_dev(old, table, offset),
                                 accumulate=True)
        assert rel_err(_host(acc), old + want_g) <= TOL[table]
        absent = np.setdiff1d(np.arange(V), ids[~masked])
        np.testing.assert_array_equal(_host(acc)[absent], old[absent])


def test_embed_empty_and_all_padding():
    import torch
    import dp_grape_projection_amd as dpg
    E = torch.randn(9, 12, device="cuda")
    assert dpg.dpg_embed(torch.empty((0, 4), dtype=torch.int64, device="cuda"), E).shape == (0, 4, 12)
    ids = torch.full((2, 3), -1, device="cuda")
    dY = torch.full((2, 3, 12), float("nan"), device="cuda")
    assert not dpg.dpg_embed(ids, E).any()
    assert not dpg.dpg_embed_grad(ids, dY, 9).any()
    norm_sq = torch.ones(2, device="cuda")
    dpg.dpg_embed_norms(ids, dY, 9, norm_sq)
    assert torch.equal(norm_sq, torch.ones(2, device="cuda"))


def test_embed_offsets_past_32_bits():
    """Table, output and gradient of more than 2^32 elements (8.6 GB each)."""
    import torch
    import dp_grape_projection_amd as dpg
    V, d = 2 ** 20 + 5, 4104
    E = torch.empty((V, d), dtype=torch.bfloat16, device="cuda")
    E.copy_((torch.arange(V, device="cuda") % 31).to(torch.bfloat16)[:, None].expand(V, d))
    ids = torch.tensor([[V - 1, 0, V - 2, 12345, V]], device="cuda")
    Y = dpg.dpg_embed(ids, E)
    want = torch.tensor([(V - 1) % 31, 0, (V - 2) % 31, 12345 % 31, 0], device="cuda")
    assert torch.equal(Y[0].float(), want.float()[:, None].expand(5, d))
    # E as the gradient of V positions: three tokens in turn, the last one absent
    pos = (torch.arange(V, device="cuda") % 3).view(1, V)
    dE = dpg.dpg_embed_grad(pos, E.view(1, V, d), 4, table_dtype=torch.float32)
    col = (torch.arange(V, device="cuda") % 31).double()
    for v in range(4):
        total = float(col[pos[0] == v].sum())
        err = (dE[v].double() - total).abs().max().item()
        assert err <= 1e-5 * max(total, 1.0), (v, err)
    # a dE whose last rows lie past 2^32 elements
    dY = torch.ones((1, 5, d), dtype=torch.bfloat16, device="cuda")
    dpg.dpg_embed_grad(ids, dY, V, dE=E)
    assert torch.equal(E[V - 1], dY[0, 0]) and torch.equal(E[12345], dY[0, 0])
    assert not E[V - 3].any() and not E[1].any()


# ----------------------------------------------------------------- losses --

# N, d, V
LOSS = [
    (1, 1, 1), (1, 8, 5), (5, 37, 100), (130, 200, 1000), (257, 64, 3001), (300, 1002, 515),
    (3, 2048, 777), (1, 64, 4100), (64, 72, 259), (520, 256, 4099), (17, 4096, 300),
]


def _loss_case(N, d, V, k, act, seed):
    r = np.random.default_rng([N, d, V, k, seed])
    E = _round(r.standard_normal((V, d)) * 2.0 / math.sqrt(d), act)
    X = _round(r.standard_normal((N, d)), act)
    ids = np.stack([r.permutation(V)[:k] if V >= k else r.integers(0, V, k) for _ in range(N)])
    off = r.random((N, k)) < 0.2
    ids[off] = r.choice([-1, V, 2 ** 40, -2 ** 40], off.sum())
    if N > 2:
        ids[1] = -1                        # a row without any target
        ids[N - 1] = V
    t = (r.standard_normal((N, k)) * 2.0).astype(np.float32)
    g = r.standard_normal(N).astype(np.float32)
    return X, E, ids, t, g


def _check_loss(X, E, ids, q, loss, lse, scale, tau):
    want, want_lse, _, _ = ot.target_loss(X, E, ids, q, scale, tau)
    bar = 2e-5 * np.maximum(1.0, np.abs(want_lse)) * max(1.0, tau * tau)
    assert (np.abs(_host(loss) - want) <= bar).all(), np.abs(_host(loss) - want).max()
    assert (np.abs(_host(lse) - want_lse) <= bar).all()


def _poison(X, ids, V):
    """X with NaN and infinities in the rows that have no target."""
    X = X.copy()
    dead = ~((ids >= 0) & (ids < V)).any(-1)
    X[dead] = np.nan
    X[dead, ::2] = np.inf
    return X


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("N,d,V", LOSS)
def test_vocab_loss(N, d, V, act):
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[vocab] N={N} d={d} V={V} {act}", flush=True)
    X, E, ids, _, g = _loss_case(N, d, V, 1, act, 1)
    ids = ids[:, 0]
    q = ((ids >= 0) & (ids < V)).astype(np.float64)
    _, _, want_dX, want_dE = ot.target_loss(X, E, ids, q, 0.8, 1.0, g)
    Xp = _poison(X, ids[:, None], V)
    gp = np.where(q > 0, g, np.float32(np.nan))
    for offset in (0, 1):
        x, e, y = _dev(Xp, act, offset), _dev(E, act, offset), _dev(ids)
        loss, lse = dpg.dpg_vocab_loss(x, e, y, scale=0.8)
        _check_loss(X, E, ids, q, loss, lse, 0.8, 1.0)
        dX, dE = dpg.dpg_vocab_loss_grad(x, e, y, lse, _dev(gp), scale=0.8)
        assert rel_err(_host(dX), want_dX) <= TOL[act]
        assert rel_err(_host(dE), want_dE) <= TOL[act]
        dX1, none = dpg.dpg_vocab_loss_grad(x, e, y, lse, _dev(gp), scale=0.8, need_dE=False)
        none2, dE1 = dpg.dpg_vocab_loss_grad(x, e, y, lse, _dev(gp), scale=0.8, need_dX=False)
        assert none is None and none2 is None
        assert torch.equal(dX, dX1) and torch.equal(dE, dE1)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("k,tau", [(1, 1.0), (7, 2.0), (64, 0.7), (100, 4.0)])
@pytest.mark.parametrize("N,d,V", [(1, 8, 5), (5, 37, 130), (130, 200, 1000), (257, 64, 3001),
                                   (40, 1002, 515)])
def test_distill_loss(N, d, V, k, tau, act):
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[distill] N={N} d={d} V={V} k={k} tau={tau} {act}", flush=True)
    X, E, ids, t, g = _loss_case(N, d, V, k, act, 2)
    if N > 6 and k > 2:
        ids[3, 1] = ids[3, 0]              # an id named twice
        ids[4, :] = 2                      # and one named k times
        t[5, 1:] = -np.inf                 # a single entry with weight
        t[6, :] = -np.inf                  # no weight at all
        t[0, 0] = np.finfo(np.float32).min
    q = ot.teacher_weights(ids, t, V, tau)
    _, _, want_dX, want_dE = ot.target_loss(X, E, ids, q, 1.2, tau, g)
    dead = ~(q > 0).any(-1)
    Xp = X.copy()
    Xp[dead] = np.nan
    for offset in (0, 1):
        x, e, y, tt = _dev(Xp, act, offset), _dev(E, act, offset), _dev(ids), _dev(t)
        loss, lse = dpg.dpg_distill_loss(x, e, y, tt, temperature=tau, scale=1.2)
        _check_loss(X, E, ids, q, loss, lse, 1.2, tau)
        dX, dE = dpg.dpg_distill_loss_grad(x, e, y, tt, lse, _dev(g), temperature=tau, scale=1.2)
        assert rel_err(_host(dX), want_dX) <= TOL[act]
        assert rel_err(_host(dE), want_dE) <= TOL[act]
        dX1, _ = dpg.dpg_distill_loss_grad(x, e, y, tt, lse, _dev(g), temperature=tau, scale=1.2,
                                           need_dE=False)
        assert torch.equal(dX, dX1)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_losses_without_any_target(act):
    import torch
    import dp_grape_projection_amd as dpg
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    X = torch.full((6, 64), float("nan"), dtype=dt, device="cuda")
    E = torch.randn(300, 64, device="cuda").to(dt)
    ids = torch.full((6,), -100, device="cuda")
    loss, lse = dpg.dpg_vocab_loss(X, E, ids)
    assert not loss.any() and not lse.any()
    dX, dE = dpg.dpg_vocab_loss_grad(X, E, ids, lse, loss)
    assert not dX.any() and not dE.any()
    top = ids[:, None].expand(6, 3).contiguous()
    t = torch.zeros(6, 3, device="cuda")
    loss, lse = dpg.dpg_distill_loss(X, E, top, t)
    dX, dE = dpg.dpg_distill_loss_grad(X, E, top, t, lse, loss)
    assert not loss.any() and not dX.any() and not dE.any()
    none = torch.empty((0, 64), dtype=dt, device="cuda")
    loss, lse = dpg.dpg_vocab_loss(none, E, ids[:0])
    dX, dE = dpg.dpg_vocab_loss_grad(none, E, ids[:0], lse, loss)
    assert loss.numel() == 0 and dX.shape == (0, 64) and not dE.any()


def test_large_logits_and_nan_stay_in_their_rows():
    """Logits of several hundred neither overflow nor lose the loss; a NaN in
    one row's X reaches that row's loss and gradient only."""
    import torch
    import dp_grape_projection_amd as dpg
    r = np.random.default_rng(5)
    X, E = r.standard_normal((9, 64)) * 40.0, r.standard_normal((777, 64))
    X, E = _round(X, "fp32"), _round(E, "fp32")
    ids = r.integers(0, 777, 9)
    loss, lse = dpg.dpg_vocab_loss(_dev(X, "fp32"), _dev(E, "fp32"), _dev(ids))
    want, want_lse, _, _ = ot.target_loss(X, E, ids, np.ones(9))
    assert want_lse.max() > 500
    assert (np.abs(_host(loss) - want) <= 2e-5 * np.abs(want_lse)).all()
    X[4, 3] = np.nan
    x = _dev(X, "fp32")
    loss2, lse2 = dpg.dpg_vocab_loss(x, _dev(E, "fp32"), _dev(ids))
    keep = [i for i in range(9) if i != 4]
    assert torch.isnan(loss2[4]) and torch.equal(loss2[keep], loss[keep])
    dX, _ = dpg.dpg_vocab_loss_grad(x, _dev(E, "fp32"), _dev(ids), lse2, torch.ones_like(loss),
                                    need_dE=False)
    assert torch.isnan(dX[4]).all() and torch.isfinite(dX[keep]).all()


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_gradient_in_several_pieces(act):
    """More rows than one piece of D takes of the vocabulary: the pieces' sums
    agree with a float64 computation over whole rows."""
    import torch
    import dp_grape_projection_amd as dpg
    N, d, V = 70000, 24, 5000
    g0 = torch.Generator(device="cuda").manual_seed(6)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    X = torch.randn(N, d, generator=g0, device="cuda").to(dt)
    E = (torch.randn(V, d, generator=g0, device="cuda") * 0.4).to(dt)
    ids = torch.randint(-V // 10, V, (N,), generator=g0, device="cuda")
    w = torch.rand(N, generator=g0, device="cuda")
    loss, lse = dpg.dpg_vocab_loss(X, E, ids)
    dX, dE = dpg.dpg_vocab_loss_grad(X, E, ids, lse, w)
    want_dE = torch.zeros((V, d), dtype=torch.float64, device="cuda")
    for n0 in range(0, N, 10000):
        sl = slice(n0, n0 + 10000)
        on = ids[sl] >= 0
        z = X[sl].double() @ E.double().t()
        p = torch.softmax(z, 1)
        at = ids[sl].clamp(min=0)[:, None]
        want = (torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]) * on
        assert (loss[sl].double() - want).abs().max().item() <= 4e-5
        D = p.scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64))
        D = D * (w[sl].double() * on)[:, None]
        assert rel_err(_host(dX[sl]), (D @ E.double()).cpu().numpy()) <= TOL[act]
        want_dE += D.t() @ X[sl].double()
    assert rel_err(_host(dE), want_dE.cpu().numpy()) <= TOL[act]


@pytest.mark.parametrize("which", ["vocab", "distill"])
def test_gradient_against_differences(which):
    """The directional derivative of the summed loss along U, by central
    differences of the fp32 loss, against <dX, U> and <dE, U>. With h = 1e-2
    the differences carry h^2 / 6 times a third derivative of order one, and
    loss errors of 1e-6 over h: together below 1e-3 of a derivative of order
    ten."""
    import torch
    import dp_grape_projection_amd as dpg
    X, E, ids, t, g = _loss_case(60, 48, 501, 5, "fp32", 9)
    x, e, tt, gg = _dev(X, "fp32"), _dev(E, "fp32"), _dev(t), _dev(np.abs(g))
    y = _dev(ids if which == "distill" else ids[:, 0])

    def total(x, e):
        if which == "vocab":
            loss, lse = dpg.dpg_vocab_loss(x, e, y)
        else:
            loss, lse = dpg.dpg_distill_loss(x, e, y, tt, temperature=1.5)
        return float((loss.double() * gg.double()).sum()), lse

    _, lse = total(x, e)
    if which == "vocab":
        dX, dE = dpg.dpg_vocab_loss_grad(x, e, y, lse, gg)
    else:
        dX, dE = dpg.dpg_distill_loss_grad(x, e, y, tt, lse, gg, temperature=1.5)
    h = 1e-2
    for dA, step in ((dX, lambda u: (x + u, e)), (dE, lambda u: (x, e + u))):
        U = dA / dA.norm()
        want = float((dA.double() * U.double()).sum())
        diff = (total(*step(h * U))[0] - total(*step(-h * U))[0]) / (2 * h)
        assert abs(diff - want) <= 1e-3 * max(abs(want), 10.0), (diff, want)


# ------------------------------------------------- streams, graphs, errors --

def test_side_stream_and_caller_buffers():
    import torch
    import dp_grape_projection_amd as dpg
    X, E, ids, _, g = _loss_case(130, 200, 1000, 1, "bf16", 4)
    x, e, y, gg = _dev(X, "bf16"), _dev(E, "bf16"), _dev(ids[:, 0]), _dev(g)
    loss0, lse0 = dpg.dpg_vocab_loss(x, e, y)
    dX0, dE0 = dpg.dpg_vocab_loss_grad(x, e, y, lse0, gg)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    loss1, lse1 = dpg.dpg_vocab_loss(x, e, y, stream=s)
    dX1, dE1 = dpg.dpg_vocab_loss_grad(x, e, y, lse1, gg, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in ((loss0, loss1), (lse0, lse1), (dX0, dX1), (dE0, dE1)):
        assert torch.equal(a, b)


def test_graph_replays():
    """The whole set captured once and replayed, with eager work in between."""
    import torch
    import dp_grape_projection_amd as dpg
    X, E, ids, _, g = _loss_case(130, 200, 1000, 1, "bf16", 4)
    x, e, y, gg = _dev(X, "bf16"), _dev(E, "bf16"), _dev(ids[:, 0]), _dev(g)
    tok = _dev(ids[:, 0].reshape(10, 13))

    def step():
        loss, lse = dpg.dpg_vocab_loss(x, e, y)
        dX, dE = dpg.dpg_vocab_loss_grad(x, e, y, lse, gg)
        n2 = torch.zeros(10, device="cuda")
        dpg.dpg_embed_norms(tok, dX.view(10, 13, 200), 1000, n2)
        dpg.dpg_embed_grad(tok, dX.view(10, 13, 200), 1000, dE=dE, accumulate=True)
        return loss, dX, dE, n2

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(_dev(X * (1.0 + 0.1 * k), "bf16"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), k


def test_binding_refusals():
    import torch
    import dp_grape_projection_amd as dpg
    X = torch.randn(4, 16, device="cuda")
    E = torch.randn(9, 16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        dpg.dpg_vocab_loss(X, E.bfloat16(), ids)
    with pytest.raises(TypeError):
        dpg.dpg_vocab_loss(X, E, ids.int())
    with pytest.raises(TypeError):
        dpg.dpg_vocab_loss(X.half(), E.half(), ids)
    with pytest.raises(ValueError):
        dpg.dpg_vocab_loss(X, E[:, :8], ids)
    with pytest.raises(ValueError):
        dpg.dpg_vocab_loss(X, E.t().contiguous(), ids)
    with pytest.raises(ValueError):
        dpg.dpg_vocab_loss(X, E, ids[:3])
    with pytest.raises(ValueError):
        dpg.dpg_vocab_loss(X.cpu(), E, ids)
    with pytest.raises(ValueError):
        dpg.dpg_vocab_loss_grad(X, E, ids, f, f, need_dX=False, need_dE=False)
    with pytest.raises(ValueError):
        dpg.dpg_vocab_loss_grad(X, E, ids, f[:2], f)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_vocab_loss(X, E, ids, scale=float("inf"))
    with pytest.raises(dpg.DpgError):
        dpg.dpg_vocab_loss(X, E, ids, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    top, t = ids.view(4, 1), f.view(4, 1)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_distill_loss(X, E, top, t, temperature=0.0)
    with pytest.raises(ValueError):
        dpg.dpg_distill_loss(X, E, top, f)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_embed(ids, E.bfloat16(), dtype=torch.float32)
    with pytest.raises(ValueError):
        dpg.dpg_embed_grad(ids.view(2, 2), X, 9)
    with pytest.raises(ValueError):
        dpg.dpg_embed_grad(ids.view(2, 2), X.view(2, 2, 16), 9, accumulate=True)
    with pytest.raises(dpg.DpgError):
        dpg.dpg_embed_grad(ids.view(2, 2), X.view(2, 2, 16), 0)


def test_distillation_id_named_with_and_without_weight():
    """An id named first with a logit of -inf and again with a finite one."""
    import dp_grape_projection_amd as dpg
    X, E, _, _, g = _loss_case(4, 64, 300, 1, "fp32", 11)
    ids = np.array([[7, 7, 9], [9, 7, 7], [7, 9, 7], [5, 5, 5]])
    t = np.array([[-np.inf, 1.0, 0.5], [0.5, -np.inf, 1.0], [1.0, 0.5, -np.inf],
                  [-np.inf, -np.inf, 2.0]], np.float32)
    q = ot.teacher_weights(ids, t, 300, 1.0)
    _, _, want_dX, want_dE = ot.target_loss(X, E, ids, q, 1.0, 1.0, g)
    x, e, y, tt = _dev(X, "fp32"), _dev(E, "fp32"), _dev(ids), _dev(t)
    loss, lse = dpg.dpg_distill_loss(x, e, y, tt)
    _check_loss(X, E, ids, q, loss, lse, 1.0, 1.0)
    dX, dE = dpg.dpg_distill_loss_grad(x, e, y, tt, lse, _dev(g))
    assert rel_err(_host(dX), want_dX) <= TOL["fp32"]
    assert rel_err(_host(dE), want_dE) <= TOL["fp32"]


def test_fp32_rows_of_very_different_size():
    """fp32 rows of X and of E of sizes from 2^-60 to 2^3, some with one
    element 2^12 above the rest. A logit is off by at most the fp32 bar of the sum
    of its products' magnitudes, and 2^-38 of either row's largest element times
    the other's sum (twice that with both); the loss by two logits' errors."""
    import torch
    import dp_grape_projection_amd as dpg
    N, d, V = 300, 72, 519
    r = np.random.default_rng(91)
    px, pe = r.integers(-60, 41, N), r.integers(-40, 61, V)
    E = r.standard_normal((V, d)) * 2.0 ** np.minimum(pe, 0)[:, None]
    X = r.standard_normal((N, d)) * 2.0 ** np.minimum(px, 3)[:, None]
    X[::3, 5] *= 2.0 ** 12
    E[::4, 5] *= 2.0 ** -10
    E[1::4, 9] *= 2.0 ** 12
    X[:, 9] *= 2.0 ** -10
    X, E = _round(X, "fp32"), _round(E, "fp32")
    y = r.integers(0, V, N)
    z = X @ E.T
    m = z.max(axis=1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(axis=1))
    loss = lse - z[np.arange(N), y]
    aX, aE = np.abs(X), np.abs(E)
    dz = (1e-5 * (aX @ aE.T) + 2.0 ** -37 * (np.outer(aX.max(1), aE.sum(1)) + np.outer(aX.sum(1), aE.max(1))))
    bar = 2 * dz.max(axis=1) + 2e-5 * np.maximum(1.0, np.abs(lse))
    print("[tokens] fp32 rows of very different size", flush=True)
    got, got_lse = dpg.dpg_vocab_loss(_dev(X, "fp32"), _dev(E, "fp32"), _dev(y))
    torch.cuda.synchronize()
    assert (np.abs(_host(got_lse) - lse) <= bar).all()
    assert (np.abs(_host(got) - loss) <= bar).all()


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("N,d,V", [(1500, 70, 300), (3000, 129, 130)])
def test_gradients_of_many_rows_and_few_columns(N, d, V, act):
    """Long sums for few outputs, which are split over blocks, into buffers that
    start one element off."""
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[vocab] many rows N={N} d={d} V={V} {act}", flush=True)
    X, E, ids, _, g = _loss_case(N, d, V, 1, act, 5)
    ids = ids[:, 0]
    q = ((ids >= 0) & (ids < V)).astype(np.float64)
    _, want_lse, want_dX, want_dE = ot.target_loss(X, E, ids, q, 1.0, 1.0, g)
    x, e, y = _dev(X, act, 1), _dev(E, act, 1), _dev(ids)
    loss, lse = dpg.dpg_vocab_loss(x, e, y)
    _check_loss(X, E, ids, q, loss, lse, 1.0, 1.0)
    dX, dE = _dev(np.full((N, d), 7.0), act, 1), _dev(np.full((V, d), 7.0), act, 1)
    out = dpg.dpg_vocab_loss_grad(x, e, y, lse, _dev(g), dX=dX, dE=dE)
    assert out[0] is dX and out[1] is dE
    assert rel_err(_host(dX), want_dX) <= TOL[act]
    assert rel_err(_host(dE), want_dE) <= TOL[act]
    again = dpg.dpg_vocab_loss_grad(x, e, y, lse, _dev(g))
    assert torch.equal(again[0], dX) and torch.equal(again[1], dE)


@pytest.mark.parametrize("N,d,V", [(128, 132, 700), (97, 260, 515), (16, 20, 130), (33, 4, 129),
                                   (64, 1000, 257), (7, 512, 5000)])
def test_few_fp32_rows(N, d, V):
    """At most 128 fp32 rows, whose table is read as it is where its rows are whole
    16 bytes, and packed otherwise (one element off): both against the reference."""
    import dp_grape_projection_amd as dpg
    print(f"[tokens] few fp32 rows N={N} d={d} V={V}", flush=True)
    X, E, ids, t, g = _loss_case(N, d, V, 6, "fp32", 7)
    y = ids[:, 0]
    q1 = ((y >= 0) & (y < V)).astype(np.float64)
    qk = ot.teacher_weights(ids, t, V, 2.0)
    _, _, dX1, dE1 = ot.target_loss(X, E, y, q1, -0.9, 1.0, g)
    _, _, dXk, dEk = ot.target_loss(X, E, ids, qk, 1.1, 2.0, g)
    Xp = _poison(X, ids, V)
    for offset in (0, 1):
        x, e = _dev(Xp, "fp32"), _dev(E, "fp32", offset)
        loss, lse = dpg.dpg_vocab_loss(x, e, _dev(y), scale=-0.9)
        on = np.flatnonzero(q1 > 0)
        _check_loss(X[on], E, y[on], q1[on], loss[on], lse[on], -0.9, 1.0)
        dX, dE = dpg.dpg_vocab_loss_grad(x, e, _dev(y), lse, _dev(g), scale=-0.9)
        assert np.isfinite(_host(dX)).all() and np.isfinite(_host(dE)).all()
        assert rel_err(_host(dX), dX1) <= TOL["fp32"]
        assert rel_err(_host(dE), dE1) <= TOL["fp32"]
        loss, lse = dpg.dpg_distill_loss(x, e, _dev(ids), _dev(t), temperature=2.0, scale=1.1)
        _check_loss(X, E, ids, qk, loss, lse, 1.1, 2.0)
        dX, dE = dpg.dpg_distill_loss_grad(x, e, _dev(ids), _dev(t), lse, _dev(g),
                                           temperature=2.0, scale=1.1)
        assert np.isfinite(_host(dX)).all() and np.isfinite(_host(dE)).all()
        assert rel_err(_host(dX), dXk) <= TOL["fp32"]
        assert rel_err(_host(dE), dEk) <= TOL["fp32"]


def test_few_fp32_rows_in_several_pieces():
    import torch
    import dp_grape_projection_amd as dpg
    N, d, V = 9, 4096, 45000
    g0 = torch.Generator(device="cuda").manual_seed(8)
    X = torch.randn(N, d, generator=g0, device="cuda")
    E = torch.randn(V, d, generator=g0, device="cuda") / 32
    y = torch.randint(0, V, (N,), generator=g0, device="cuda")
    y[3] = -1
    w = torch.rand(N, generator=g0, device="cuda")
    loss, lse = dpg.dpg_vocab_loss(X, E, y)
    dX, dE = dpg.dpg_vocab_loss_grad(X, E, y, lse, w)
    on = (y >= 0).double()
    z = X.double() @ E.double().t()
    want = (torch.logsumexp(z, 1) - z.gather(1, y.clamp(min=0)[:, None])[:, 0]) * on
    assert (loss.double() - want).abs().max().item() <= 4e-5
    D = torch.softmax(z, 1).scatter_add(1, y.clamp(min=0)[:, None],
                                        -torch.ones((N, 1), dtype=torch.float64, device="cuda"))
    D = D * (w.double() * on)[:, None]
    assert rel_err(_host(dX), (D @ E.double()).cpu().numpy()) <= TOL["fp32"]
    err = (dE.double() - D.t() @ X.double()).norm() / (D.t() @ X.double()).norm()
    assert err.item() <= TOL["fp32"]


@pytest.mark.parametrize("N,d,V", [(128, 1028, 8200), (97, 260, 33000), (33, 4100, 2050),
                                   (16, 1000, 8500), (65, 1024, 8193), (64, 516, 16500)])
def test_few_fp32_rows_of_a_large_table(N, d, V):
    """A table large enough to be read as it is, against float64; one element off,
    where it is packed, it meets the same bars."""
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[tokens] few fp32 rows, large table N={N} d={d} V={V}", flush=True)
    g0 = torch.Generator(device="cuda").manual_seed(9)
    X = torch.randn(N, d, generator=g0, device="cuda")
    E = torch.randn(V, d, generator=g0, device="cuda") * 2 / math.sqrt(d)
    k = 5
    ids = torch.randint(-V // 8, V, (N, k), generator=g0, device="cuda")
    ids[N // 2] = -1
    X[N // 2] = float("nan")                  # a row without target
    t = torch.randn(N, k, generator=g0, device="cuda") * 2
    w = torch.rand(N, generator=g0, device="cuda")
    E1 = torch.empty(V * d + 1, device="cuda")[1:].view(V, d).copy_(E)
    got, off = [], []
    for e, out in ((E, got), (E1, off)):
        out.extend(dpg.dpg_distill_loss(X, e, ids, t, temperature=2.0))
        out.extend(dpg.dpg_distill_loss_grad(X, e, ids, t, out[1], w, temperature=2.0))
    valid = ids >= 0
    on = valid.any(1)
    Xd = torch.where(on[:, None], X, 0.0).double()
    z = Xd @ E.double().t() / 2
    q = torch.where(valid, t.double() / 2, -math.inf).softmax(1).nan_to_num(0.0)
    dist = torch.zeros_like(z).scatter_add(1, ids.clamp(min=0), q)
    lse = torch.logsumexp(z, 1)
    loss = 4 * (torch.xlogy(q, q).sum(1) - (dist * z).sum(1) + lse) * on
    D = (z.softmax(1) - dist) * (w.double() * 2 * on)[:, None]
    want = [loss, lse * on, D @ E.double(), D.t() @ Xd]
    bar = 2e-5 * max(1.0, lse.abs().max().item()) * 4
    for a, b, c in zip(got, off, want):
        assert torch.isfinite(a).all() and torch.isfinite(b).all()
        if a.dim() == 1:
            assert (a.double() - c).abs().max().item() <= bar
            assert (b.double() - c).abs().max().item() <= bar
        else:
            assert rel_err(_host(a), c.cpu().numpy()) <= TOL["fp32"]
            assert rel_err(_host(b), c.cpu().numpy()) <= TOL["fp32"]


def test_few_fp32_rows_of_an_unaligned_table_in_pieces():
    """One element off, a table is packed 64 MiB at a time."""
    import torch
    import dp_grape_projection_amd as dpg
    N, d, V = 5, 1000, 30000
    g0 = torch.Generator(device="cuda").manual_seed(10)
    X = torch.randn(N, d, generator=g0, device="cuda")
    E = torch.randn(V * d + 1, generator=g0, device="cuda")[1:].view(V, d)
    y = torch.tensor([0, 29999, -1, 15000, 11008], device="cuda")
    w = torch.rand(N, generator=g0, device="cuda")
    loss, lse = dpg.dpg_vocab_loss(X, E, y, scale=0.05)
    dX, dE = dpg.dpg_vocab_loss_grad(X, E, y, lse, w, scale=0.05)
    on = (y >= 0).double()
    z = 0.05 * (X.double() @ E.double().t())
    at = y.clamp(min=0)[:, None]
    want = (torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]) * on
    assert (loss.double() - want).abs().max().item() <= 4e-5 * max(1.0, want.max().item())
    D = torch.softmax(z, 1).scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64))
    D = D * (0.05 * w.double() * on)[:, None]
    assert torch.isfinite(dX).all() and torch.isfinite(dE).all()
    assert rel_err(_host(dX), (D @ E.double()).cpu().numpy()) <= TOL["fp32"]
    assert rel_err(_host(dE), (D.t() @ X.double()).cpu().numpy()) <= TOL["fp32"]


@pytest.mark.parametrize("N,d,V", [(129, 1024, 8300), (500, 260, 33000), (385, 4100, 2050)])
def test_fp32_gradients_of_a_few_hundred_rows(N, d, V):
    """dX from a table read as it is, and from a packed one (one element off)."""
    import torch
    import dp_grape_projection_amd as dpg
    print(f"[tokens] a few hundred fp32 rows N={N} d={d} V={V}", flush=True)
    g0 = torch.Generator(device="cuda").manual_seed(11)
    X = torch.randn(N, d, generator=g0, device="cuda")
    E = torch.randn(V, d, generator=g0, device="cuda") * 2 / math.sqrt(d)
    E1 = torch.empty(V * d + 1, device="cuda")[1:].view(V, d).copy_(E)
    y = torch.randint(-V // 8, V, (N,), generator=g0, device="cuda")
    w = torch.rand(N, generator=g0, device="cuda")
    on = (y >= 0).double()[:, None]
    D = (X.double() @ E.double().t()).softmax(1)
    D = D.scatter_add(1, y.clamp(min=0)[:, None], -torch.ones_like(on)) * w.double()[:, None] * on
    want_dX, want_dE = (D @ E.double()).cpu().numpy(), (D.t() @ X.double()).cpu().numpy()
    for e in (E, E1):
        _, lse = dpg.dpg_vocab_loss(X, e, y)
        dX, dE = dpg.dpg_vocab_loss_grad(X, e, y, lse, w)
        only, _ = dpg.dpg_vocab_loss_grad(X, e, y, lse, w, need_dE=False)
        assert torch.isfinite(dX).all() and torch.isfinite(dE).all() and torch.equal(dX, only)
        assert rel_err(_host(dX), want_dX) <= TOL["fp32"]
        assert rel_err(_host(dE), want_dE) <= TOL["fp32"]
