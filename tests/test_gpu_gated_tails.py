"""The gated block's activations value by value, relative to each value, from where they
vanish to where they are the identity, and where a gate is no number.

The gate of row n is g_n in every column and the up projection 1 (products of exact parts
by ones and zeros), W_out the identity and dY ones: H is act(g), dU is act(g) and dG is
act'(g), each rounded once.

Tolerances, with u = 2^-24. e^t is taken of an argument that is rounded (by 1.5 u with the
constant's own rounding), so it is off by 1.5 |t| u, and the instruction by 2 u.
  silu      x s, s = 1 / (1 + e^-x): (1.5 |x| + 8) u; the slope s (1 + x (1 - s)) loses as
            much of s (1 + |x|), where 1 - s is off by u itself.
  gelu      x Phi(x): the argument of the tail, off by 1.5 u of itself, moves Phi by
            (x^2 + 1) 1.5 u, and 16 last places of the function are 32 u; the slope loses
            as much of Phi + |x| phi, whose exponent x^2 / 2 has two roundings.
  gelu tanh x s(t), t = 2 sqrt(2 / pi) (x + 0.044715 x^3): t is off by 6 u of itself, hence
            (7.5 |t| + 8) u; the slope loses as much of s + |x| s (1 - s) t'(x), and 4 u of
            s |x| t'(x) where 1 - s cancels.
bf16 rounds the result by 2^-8 at most."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U, D = 2.0 ** -24, 32
REACH = {"silu": 80.0, "gelu": 12.0, "gelu_tanh": 9.5}


@pytest.fixture(scope="module", autouse=True)
def gpu_and_library():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dp_grape_projection_amd as dpg
    dpg.load_library()     # fails loudly when libdpg.so is missing


def _truth(x, act):
    """act(x), act'(x) and what either may be off by in fp32."""
    a = np.abs(x)
    if act == "silu":
        s = np.where(x < 0, np.exp(-a), 1.0) / (1.0 + np.exp(-a))
        e = (1.5 * a + 8) * U
        return x * s, s * (1 + x * (1 - s)), a * s * e, 2 * s * (1 + a) * e
    if act == "gelu":
        cdf = 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0))
        phi = np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        e = (1.5 * (a * a + 1) + 36) * U
        return x * cdf, cdf + x * phi, a * cdf * e, (cdf + a * phi) * e
    c = 2 * math.sqrt(2 / math.pi)
    t, dt = c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x)
    p = np.exp(-np.abs(t))
    s, r = np.where(t < 0, p, 1.0) / (1 + p), np.where(t < 0, 1.0, p) / (1 + p)
    e = (7.5 * np.abs(t) + 8) * U
    return (x * s, s + x * s * r * dt, a * s * e,
            2 * (s + a * s * r * dt) * e + 4 * U * s * a * dt)


def _operands(gates, dtype):
    import torch
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    N = len(gates)
    X = torch.zeros(N, D, device="cuda", dtype=dt)
    X[:, 0] = torch.from_numpy(gates).to("cuda", dt)
    X[:, 1] = 1
    W_in = torch.zeros(D, 2 * D, device="cuda", dtype=dt)
    W_in[0, :D], W_in[1, D:] = 1, 1
    return X, W_in, torch.eye(D, device="cuda", dtype=dt), torch.ones(N, D, device="cuda", dtype=dt)


def _close(got, want, off, dtype, name):
    got = got.double().cpu().numpy()
    assert got.shape == (len(want), D)
    off = off + (2.0 ** -8 * (np.abs(want) + off) if dtype == "bf16" else 0.0)
    worst = np.abs(got - want[:, None]) / (off[:, None] + 1e-300)
    at = np.unravel_index(np.argmax(worst), worst.shape)
    assert worst[at] <= 1, (name, at[0], got[at], want[at[0]], worst[at])


# a kernel of few rows (bf16), tiles whose H is kept in two parts, and tiles
@pytest.mark.parametrize("N", [16, 60, 300])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_every_value_to_its_own_precision(act, dtype, N):
    import dp_grape_projection_amd as dpg
    print(f"[tails] {act} {dtype} {N}", flush=True)
    gates = np.linspace(-REACH[act], REACH[act], N).astype(np.float32)
    X, W_in, W_out, dY = _operands(gates, dtype)
    x = X[:, 0].double().cpu().numpy()
    value, slope, off, off_slope = _truth(x, act)
    Y, Z = dpg.dpg_gated(X, W_in, W_out, act=act, keep=True)
    _close(Y, value, off, dtype, "Y")
    kept = dpg.dpg_unpack_act(Z).double().cpu().numpy()
    assert (kept[:, 0] == kept[:, 0, :1]).all() and (kept[:, 1] == 1).all()
    for name, z, at in (("again", None, x), ("codes", Z, kept[:, 0, 0])):
        value, slope, off, off_slope = _truth(at, act)
        g = dpg.dpg_gated_grad(dY, X, W_in, W_out, act=act, Z=z, need_dW=False, need_layers=True)
        _close(g.H, value, off, dtype, name + " H")
        _close(g.dZ[:, D:], value, off, dtype, name + " dU")
        _close(g.dZ[:, :D], slope, off_slope, dtype, name + " dG")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_a_gate_that_is_no_number(act, dtype):
    """What was kept of G reads as NaN in some blocks of 32 columns, U does not: H, dU and
    dG are NaN there, and nowhere else."""
    import torch
    import dp_grape_projection_amd as dpg
    for N in (40, 200):
        X, W_in, W_out, dY = _operands(np.linspace(-2, 2, N).astype(np.float32), dtype)
        _, Z = dpg.dpg_gated(X, W_in, W_out, act=act, keep=True)
        bad = torch.zeros(N, dtype=torch.bool, device="cuda")
        bad[3], bad[N - 1] = True, True
        Z.exps[bad, 0] = 255
        g = dpg.dpg_gated_grad(dY, X, W_in, W_out, act=act, Z=Z, need_layers=True)
        for t in (g.H, g.dZ[:, :D], g.dZ[:, D:]):
            assert torch.equal(t.isnan(), bad[:, None].expand(N, D))
        # (row 0 of W_in is the gates': a sum over all rows of what is NaN in some)
        assert g.dX[bad].isnan().all() and not g.dX[~bad].isnan().any()
        assert g.dW_in.isnan().all() and g.dW_out.isnan().all()
