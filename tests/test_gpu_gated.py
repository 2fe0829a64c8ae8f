"""GPU parity of the gated feed-forward block (dpg_gated, dpg_gated_grad) against the
float64 reference oracle.feedforward, at small and ragged sizes, with every kind of tile,
unaligned operands and workspaces full of NaN.

Tolerances. bf16 rounds H (or dZ) once, by at most u = 2^-8 of each value, and the output
once, by as much: element by element the error is at most u |out| + u |H| |W| (1 + u), the
second term a sum of magnitudes, to which fp32 sums of K products and an activation of a
few fp32 roundings add at most (K + 16) 2^-24 of such sums; over a whole tensor the
roundings are independent, at most u / sqrt(3) each in the mean square (the worst place
of a mantissa), which leaves 0.82 u in all: u is the bound there. fp32: 1e-5 by pieces,
the fp32 bar of the other operators (products of exact parts, sums in fp32)."""
import numpy as np
import pytest

from _helpers import rel_err, rel_fro
from oracle import feedforward as of

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _dev(a, dtype, offset=0):
    """A contiguous device copy; offset elements off an aligned start."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    flat = torch.empty(t.numel() + offset, dtype=_dtype(dtype), device="cuda")
    out = flat[offset:].view(t.shape)
    out.copy_(t)
    return out


def _host(t):
    return t.double().cpu().numpy()


def _case(N, d, f, dtype, seed=0, offset=0):
    r = np.random.default_rng([N, d, f, seed])
    X = r.standard_normal((N, d)) * np.exp(r.uniform(-1, 1, (1, d)))
    X[r.random(N) < 0.1] = 0.0                # padded positions
    dY = r.standard_normal((N, d)) * (X[:, :1] != 0) / np.sqrt(N * d)
    W_in, W_out = r.standard_normal((d, 2 * f)) / np.sqrt(d), r.standard_normal((f, d)) / np.sqrt(f)
    return [_dev(t, dtype, offset) for t in (X, W_in, W_out, dY)]


def _poisoned(need):
    import torch
    return torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN throughout


def _check(got, want, name, dtype, rounded=None):
    """rounded: sums of magnitudes of the products whose one factor was rounded to bf16
    (None: none was), and K of those sums."""
    got = _host(got)
    assert np.isfinite(got).all(), name
    if dtype == "fp32":
        assert rel_err(got, want) <= 1e-5, (name, rel_err(got, want))
        return
    bound = U * np.abs(want)
    if rounded is not None:
        sums, K = rounded
        bound = bound + sums * (U * (1 + U) + (K + 16) * 2.0 ** -24)
    else:
        bound = bound + 1e-5 * np.abs(want).max(axis=1, keepdims=True)
    assert (np.abs(got - want) <= bound + 1e-30).all(), name
    assert rel_fro(got, want) <= U, (name, rel_fro(got, want))


def _run(N, d, f, dtype, act, offset=0):
    import torch
    import dp_grape_projection_amd as dpg
    from dp_grape_projection_amd import binding as b
    X, W_in, W_out, dY = _case(N, d, f, dtype, 1, offset)
    x, wi, wo, dy = (_host(t) for t in (X, W_in, W_out, dY))
    code = b._dtype_code(X.dtype)
    ws = _poisoned(b._gated_workspace_size(N, d, f, code, int(offset > 0)))
    want, G, Uv = of.gated(x, wi, wo, act)
    H = of.activation(G, act)[0] * Uv
    Y, none = dpg.dpg_gated(X, W_in, W_out, act=act, workspace=ws)
    assert none is None
    _check(Y, want, "Y", dtype, (np.abs(H) @ np.abs(wo), f))
    Y2, Z = dpg.dpg_gated(X, W_in, W_out, act=act, keep=True)
    assert torch.equal(Y, Y2)
    # codes: within half a step of the value and its fp32 error, a whole one at 127
    zc, ze = (t.cpu().numpy().reshape(2 * N, -1) for t in (Z.codes, Z.exps))
    kept = of.unpack8(zc, ze, f).reshape(N, 2, f)
    assert not zc[:, f:].any()
    step = np.repeat(np.ldexp(1.0, ze.astype(np.int64) - 133), 32, axis=1)[:, :f].reshape(N, 2, f)
    exact = np.stack([G, Uv], 1)
    noise = ((np.abs(x) @ np.abs(wi)).reshape(N, 2, f)) * ((d + 16) * 2.0 ** -24)
    half = np.where(np.abs(exact) > 126.9 * step, 1.0, 0.5) * step
    assert (np.abs(kept - exact) <= half + noise).all()
    # the backward pass: from the codes, and with both projections computed again
    for name, Zp, Xp, g, u in (("codes", Z, X, kept[:, 0], kept[:, 1]), ("again", None, X, G, Uv)):
        ws = _poisoned(b._gated_grad_workspace_size(N, d, f, code, int(Zp is not None), 1, 1,
                                                    int(offset > 0)))
        out = dpg.dpg_gated_grad(dY, Xp, W_in, W_out, act=act, Z=Zp, need_layers=True, workspace=ws)
        dX, dWi, dWo, dZ, Hk = of.gated_grad(dy, x, g, u, wi, wo, act)
        _check(out.dZ, dZ, name + " dZ", dtype)
        _check(out.H, Hk, name + " H", dtype)
        _check(out.dX, dX, name + " dX", dtype, (np.abs(dZ) @ np.abs(wi).T, 2 * f))
        _check(out.dW_in, dWi, name + " dW_in", dtype, (np.abs(x).T @ np.abs(dZ), N))
        _check(out.dW_out, dWo, name + " dW_out", dtype, (np.abs(Hk).T @ np.abs(dy), N))
        again = dpg.dpg_gated_grad(dY, Xp, W_in, W_out, act=act, Z=Zp, need_layers=True)
        for p, q in zip(out, again):
            assert torch.equal(p, q), name
        # one output at a time gives the same
        for kw, k in ((dict(need_dX=True, need_dW=False), 0), (dict(need_dX=False, need_dW=(True, False)), 1),
                      (dict(need_dX=False, need_dW=(False, True)), 2),
                      (dict(need_dX=False, need_dW=False, need_layers=True), 3)):
            one = dpg.dpg_gated_grad(dY, Xp, W_in, W_out, act=act, Z=Zp, **kw)
            assert torch.equal(one[k], out[k]), (name, kw)
            assert [i for i, t in enumerate(one) if t is not None] == ([3, 4] if k == 3 else [k])
    # X in 8 bits, for dW_in alone
    Xp = dpg.dpg_pack_act(X)
    out = dpg.dpg_gated_grad(dY, Xp, W_in, W_out, act=act, Z=Z)
    x8 = _host(dpg.dpg_unpack_act(Xp))
    dX, dWi, dWo, dZ, Hk = of.gated_grad(dy, x8, kept[:, 0], kept[:, 1], wi, wo, act)
    _check(out.dX, dX, "8 bits dX", dtype, (np.abs(dZ) @ np.abs(wi).T, 2 * f))
    _check(out.dW_in, dWi, "8 bits dW_in", dtype, (np.abs(x8).T @ np.abs(dZ), N))


SIZES = [(1, 8, 8), (1, 1, 1), (3, 5, 7), (2, 64, 31), (4, 64, 128), (128, 64, 256), (65, 128, 96),
         (130, 100, 70), (257, 72, 264), (300, 130, 33), (64, 320, 64), (513, 65, 161),
         # few rows: one and sixteen of them, columns and K that end inside a block's
         (1, 32, 32), (16, 96, 160), (5, 2080, 1056), (16, 64, 8224), (17, 96, 160)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d,f", SIZES)
def test_block(N, d, f, dtype):
    print(f"[gated] {N} x {d} x {f} {dtype}", flush=True)
    _run(N, d, f, dtype, ("silu", "gelu", "gelu_tanh")[(N + d + f) % 3])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations(act):
    _run(70, 48, 40, "bf16", act)
    _run(70, 48, 40, "fp32", act)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unaligned_operands(dtype):
    """Rows that could be copied as they are, from an address that cannot."""
    _run(130, 64, 64, dtype, "silu", offset=1)
    _run(9, 64, 64, dtype, "gelu", offset=1)


# the tiles of 128 and of 256 rows: enough of them for the rule to take each
@pytest.mark.parametrize("N,d,f", [(520, 64, 4200), (1000, 72, 6100), (2100, 64, 520),
                                   (300, 2000, 136), (1536, 640, 2048)])
def test_larger_tiles(N, d, f):
    print(f"[gated] {N} x {d} x {f}", flush=True)
    _run(N, d, f, "bf16", "silu")


def test_larger_tiles_fp32():
    _run(1000, 72, 3100, "fp32", "gelu")


def test_runs_of_rows():
    """More tiles than the chip holds at once, their projections computed again: rows from
    the beginning, the middle and the end against calls of those rows alone."""
    import torch
    import dp_grape_projection_amd as dpg
    N, d, f = 8192 + 256 + 7, 64, 4096
    X, W_in, W_out, dY = _case(N, d, f, "bf16", 3)
    whole = dpg.dpg_gated_grad(dY, X, W_in, W_out, need_layers=True)
    for n0, n1 in ((0, 300), (8192 - 100, 8192 + 100), (8400, N)):
        part = dpg.dpg_gated_grad(dY[n0:n1].contiguous(), X[n0:n1].contiguous(), W_in, W_out,
                                  need_dW=False, need_layers=True)
        # (other tiles sum K in the same order)
        assert torch.equal(part.dZ, whole.dZ[n0:n1])
        assert torch.equal(part.H, whole.H[n0:n1])
        assert rel_fro(_host(part.dX), _host(whole.dX[n0:n1])) <= U
    want = _host(X).T @ _host(whole.dZ)
    assert rel_fro(_host(whole.dW_in), want) <= U      # (dZ as it was rounded)
    assert rel_fro(_host(whole.dW_out), _host(whole.H).T @ _host(dY)) <= U


def test_private_layers_alone_need_no_copies_of_them():
    """dZ and H written straight to the caller, their products reading them there."""
    import torch
    import dp_grape_projection_amd as dpg
    X, W_in, W_out, dY = _case(192, 64, 128, "bf16", 11)
    _, Z = dpg.dpg_gated(X, W_in, W_out, keep=True)
    for z in (None, Z):
        own = dpg.dpg_gated_grad(dY, X, W_in, W_out, Z=z, need_layers=True)
        part = dpg.dpg_gated_grad(dY, X, W_in, W_out, Z=z)
        for a, b in zip(own[:3], part[:3]):
            assert torch.equal(a, b)


def test_at_once_on_two_streams():
    """Two calls in flight at once, each with its own workspace and outputs."""
    import torch
    import dp_grape_projection_amd as dpg
    ins = [_case(1500, 256, 512, "bf16", 20 + k) for k in range(2)]
    want = [dpg.dpg_gated_grad(t[3], *t[:3], need_layers=True) for t in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[] for _ in ins]
    for _ in range(5):
        for k, (t, s) in enumerate(zip(ins, streams)):
            got[k].append(dpg.dpg_gated_grad(t[3], *t[:3], need_layers=True, stream=s))
    torch.cuda.synchronize()
    for k in range(2):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[k]))


def test_wide_values():
    """Gates of both signs far beyond where the activations saturate."""
    import torch
    import dp_grape_projection_amd as dpg
    for act in ("silu", "gelu", "gelu_tanh"):
        for scale in (30.0, 1e4, 1e18):
            X = torch.eye(16, device="cuda")
            W_in = torch.cat([torch.linspace(-scale, scale, 16 * 8, device="cuda").view(16, 8),
                              torch.ones(16, 8, device="cuda")], 1).contiguous()
            W_out = torch.eye(8, 16, device="cuda").contiguous()
            dY = torch.ones(16, 16, device="cuda")
            Y, _ = dpg.dpg_gated(X, W_in, W_out, act=act)
            g = dpg.dpg_gated_grad(dY, X, W_in, W_out, act=act, need_layers=True)
            x, wi, wo, dy = (_host(t) for t in (X, W_in, W_out, dY))
            want, G, Uv = of.gated(x, wi, wo, act)
            with np.errstate(over="ignore", invalid="ignore"):
                grads = of.gated_grad(dy, x, G, Uv, wi, wo, act)
            assert np.abs(_host(Y) - want).max() <= 1e-6 * scale
            assert np.abs(_host(g.dZ) - np.nan_to_num(grads[3])).max() <= 1e-6 * scale


def test_infinities_and_nan_stay_in_their_rows():
    import torch
    import dp_grape_projection_amd as dpg
    X, W_in, W_out, dY = _case(40, 64, 64, "bf16", 5)
    good, _ = dpg.dpg_gated(X, W_in, W_out)
    base = dpg.dpg_gated_grad(dY, X, W_in, W_out, need_dW=False, need_layers=True)
    X2 = X.clone()
    X2[7, 3], X2[20, 5] = float("nan"), float("inf")
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[7] = rows[20] = False
    Y, Z = dpg.dpg_gated(X2, W_in, W_out, keep=True)
    assert torch.equal(Y[rows], good[rows]) and Y[7].isnan().all()
    assert (Z.exps[7] == 255).all() and not Z.codes[7].any()
    for z in (None, Z):
        g = dpg.dpg_gated_grad(dY, X2, W_in, W_out, Z=z, need_dW=False, need_layers=True)
        assert g.dZ[7].isnan().all() and g.dX[7].isnan().all()
        if z is None:
            assert torch.equal(g.dX[rows], base.dX[rows]) and torch.equal(g.dZ[rows], base.dZ[rows])


def test_empty_and_refusals():
    import torch
    import dp_grape_projection_amd as dpg
    X, W_in, W_out, dY = _case(6, 16, 24, "bf16", 6)
    e = X[:0]
    Y, Z = dpg.dpg_gated(e, W_in, W_out, keep=True)
    assert tuple(Y.shape) == (0, 16) and tuple(Z.shape) == (0, 2, 24)
    g = dpg.dpg_gated_grad(e, e, W_in, W_out, need_layers=True)
    assert not g.dW_in.any() and not g.dW_out.any() and tuple(g.dZ.shape) == (0, 48)
    lead = dpg.dpg_gated(X.view(2, 3, 16), W_in, W_out, keep=True)
    assert tuple(lead[0].shape) == (2, 3, 16) and tuple(lead[1].shape) == (2, 3, 2, 24)
    _, Z = dpg.dpg_gated(X, W_in, W_out, keep=True)
    p = dpg.dpg_pack_act(X)
    for args, kw in (((X, W_in[:, :24].contiguous(), W_out), {}), ((X, W_in, W_out.t()), {}),
                     ((X[:, :8].contiguous(), W_in, W_out), {}), ((X, W_in, W_out), dict(act="relu")),
                     ((X, W_in, W_out), dict(Z=Z)), ((X, W_in, W_out), dict(Y=e))):
        with pytest.raises(ValueError):
            dpg.dpg_gated(*args, **kw)
    with pytest.raises(TypeError):
        dpg.dpg_gated(X, W_in.float(), W_out)
    with pytest.raises(TypeError):
        dpg.dpg_gated(X.half(), W_in.half(), W_out.half())
    for args, kw in (((dY, p, W_in, W_out), {}), ((dY, None, W_in, W_out), {}),
                     ((dY, None, W_in, W_out), dict(Z=Z)), ((dY, X[:3], W_in, W_out), {}),
                     ((dY, X, W_in, W_out), dict(need_dX=False, need_dW=False)),
                     ((dY[:3], X[:3], W_in, W_out), dict(Z=Z))):
        with pytest.raises(ValueError):
            dpg.dpg_gated_grad(*args, **kw)
    with pytest.raises(TypeError):
        dpg.dpg_gated_grad(dY, X.float(), W_in, W_out)
    out = dpg.dpg_gated_grad(dY, None, W_in, W_out, Z=Z, need_dW=(False, True))
    assert out.dW_in is None and out.dW_out is not None
    for bad in (X[:, :0].contiguous(),):
        with pytest.raises(dpg.DpgError):
            dpg.dpg_gated(bad, W_in[:0].contiguous(), W_out[:, :0].contiguous())
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(dpg.DpgError, match="workspace"):
        dpg.dpg_gated(X, W_in, W_out, workspace=ws)


def test_a_captured_step_replays():
    """Forward and backward in one graph, replayed on new data between eager work; two
    graphs with their own workspaces."""
    import torch
    import dp_grape_projection_amd as dpg
    s = torch.cuda.Stream()
    ins = [_case(100, 64, 96, "bf16", k) for k in (7, 8, 9)]
    X, W_in, W_out, dY = (t.clone() for t in ins[0])
    for t in (1, 2):
        dpg.dpg_gated_grad(dY, X, W_in, W_out, need_layers=True)
    graphs = []
    for int8 in (True, False):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            Y, Z = dpg.dpg_gated(X, W_in, W_out, keep=int8)
            out = dpg.dpg_gated_grad(dY, X, W_in, W_out, Z=Z, need_layers=True)
        graphs.append((graph, int8, [Y, *out]))
    for data in ins + ins[:1]:
        for dst, src in zip((X, W_in, W_out, dY), data):
            dst.copy_(src)
        for graph, int8, got in graphs:
            for t in got:
                t.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for graph, int8, got in graphs:
            Y, Z = dpg.dpg_gated(*data[:3], keep=int8)
            want = [Y, *dpg.dpg_gated_grad(data[3], *data[:3], Z=Z, need_layers=True)]
            for p, q in zip(got, want):
                assert torch.equal(p, q)
