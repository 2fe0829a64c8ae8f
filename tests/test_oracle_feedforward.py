"""The float64 reference of the gated block and of 8-bit activations, pinned by
independent checks: central differences, torch's activations in float64, and the
definition of a code applied value by value in exact arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import feedforward as of


@pytest.mark.parametrize("act,fn", [
    ("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu),
    ("gelu_tanh", lambda x: torch.nn.functional.gelu(x, approximate="tanh"))])
def test_activations(act, fn):
    x = torch.cat([torch.linspace(-30, 30, 2001, dtype=torch.float64),
                   torch.tensor([0.0, -1e-30, 1e-30])]).requires_grad_()
    y = fn(x)
    (dy,) = torch.autograd.grad(y.sum(), x)
    value, slope = of.activation(x.detach().numpy(), act)
    np.testing.assert_allclose(value, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(slope, dy.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(act):
    r = np.random.default_rng(1)
    X, W_in, W_out = r.standard_normal((5, 4)), r.standard_normal((4, 6)), r.standard_normal((3, 4))
    dY = r.standard_normal((5, 4))
    _, G, U = of.gated(X, W_in, W_out, act)
    grads = of.gated_grad(dY, X, G, U, W_in, W_out, act)
    h = 1e-6
    for i, t in enumerate((X, W_in, W_out)):
        for at in np.ndindex(*t.shape):
            old, side = t[at], []
            for s in (h, -h):
                t[at] = old + s
                side.append(np.sum(dY * of.gated(X, W_in, W_out, act)[0]))
            t[at] = old
            # error of a central difference: h^2 third derivatives, and 1e-16 / h
            assert abs((side[0] - side[1]) / (2 * h) - grads[i][at]) < 1e-7
    f = W_out.shape[0]
    np.testing.assert_allclose(grads[0], grads[3] @ W_in.T)
    np.testing.assert_allclose(grads[4], of.activation(G, act)[0] * U)
    assert grads[3].shape == (5, 2 * f)


def test_codes_are_the_definition():
    r = np.random.default_rng(2)
    x = (r.standard_normal((40, 70)) * np.exp(r.uniform(-60, 60, (40, 1)))).astype(np.float32)
    x[3] = 0.0
    x[4, :33] = [2.0 ** -149, -2.0 ** -130] + [0.0] * 31
    x[5, 40] = 3.4028235e38
    x[6, :32] = np.arange(32) * 0.5                # ties: halves of a step at 2^-2 of the top
    codes, exps = of.pack8(x)
    back = of.unpack8(codes, exps, 70)
    assert codes.shape == (40, 96) and exps.shape == (40, 3) and not codes[:, 70:].any()
    for n in range(40):
        for j in range(3):
            block = [Fraction(float(v)) for v in x[n, 32 * j:32 * (j + 1)]]
            top = max(abs(v) for v in block)
            e = -127                                # exponent field 0
            while e < 127 and top >= Fraction(2) ** (e + 1):
                e += 1
            b = max(7, e + 127)
            assert exps[n, j] == b
            step = Fraction(2) ** (b - 133)
            for i, v in enumerate(block):
                q = max(-127, min(127, round(v / step)))   # (ties to even)
                assert codes[n, 32 * j + i] == q
                assert Fraction(back[n, 32 * j + i]) == q * step
                assert abs(q * step - v) <= (step if abs(v) > 127 * step else step / 2)


def test_blocks_with_an_infinity_or_nan():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    codes, exps = of.pack8(x)
    back = of.unpack8(codes, exps, 64)
    assert exps.tolist() == [[255, 127], [127, 255]]
    assert np.isnan(back[0, :32]).all() and np.isnan(back[1, 32:]).all()
    np.testing.assert_array_equal(back[0, 32:], 1.0)


def test_every_value_is_a_bf16_number():
    codes = np.tile(np.arange(-127, 128, dtype=np.int8), (1, 1))
    codes = np.pad(codes, ((0, 0), (0, 1)))
    for b in (7, 8, 100, 200, 254):
        v = of.unpack8(codes, np.full((1, 8), b, np.uint8), 255)
        t = torch.from_numpy(v)
        assert torch.equal(t.float().bfloat16().double(), t)
