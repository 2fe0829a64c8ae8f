"""Float64 reference of the gated feed-forward block with its gradients, and of
activations in 8 bits, written from the formulas; no code is shared with the GPU path.

Parity status: pinned by tests/test_oracle_feedforward.py (differences of the forward
pass, torch's activations in float64, the definition of a code value by value).
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["pack8", "unpack8", "activation", "gated", "gated_grad"]

BLOCK = 32


def pack8(x):
    """(codes, exps) of rows x [N, d]: per block of 32 channels b = max(7, exponent field
    of the largest magnitude as fp32), q = clamp(round(x 2^(133 - b)), -127, 127), ties to
    even; a block with an infinity or NaN has b = 255 and codes of zero."""
    x = np.asarray(x, np.float64)
    N, d = x.shape
    blocks = -(-d // BLOCK)
    codes = np.zeros((N, BLOCK * blocks), np.int8)
    exps = np.zeros((N, blocks), np.uint8)
    for j in range(blocks):
        v = x[:, BLOCK * j:BLOCK * (j + 1)]
        fine = np.isfinite(v).all(1)
        top = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0.0)).max(1), 1.0)
        # m 2^e with m in [0.5, 1): the exponent field is e + 126
        b = np.maximum(7, np.where(top > 0, np.frexp(top)[1] + 126, 0))
        q = np.clip(np.rint(np.ldexp(np.where(fine[:, None], v, 0.0), (133 - b)[:, None])), -127, 127)
        codes[:, BLOCK * j:BLOCK * j + v.shape[1]] = q.astype(np.int8)
        exps[:, j] = np.where(fine, b, 255)
    return codes, exps


def unpack8(codes, exps, d):
    """What the codes stand for, [N, d]."""
    step = np.where(exps == 255, np.nan, np.ldexp(1.0, np.maximum(exps, 7).astype(np.int64) - 133))
    return (codes.astype(np.float64) * np.repeat(step, BLOCK, axis=1))[:, :d]


_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(x, act):
    """act(x) and its derivative."""
    x = np.asarray(x, np.float64)
    if act == "silu":
        s = 0.5 * (1.0 + np.tanh(0.5 * x))
        return x * s, s + x * s * (1.0 - s)
    if act == "gelu":
        cdf = 0.5 * (1.0 + _erf(x / math.sqrt(2.0)))
        return x * cdf, cdf + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (
        1.0 + 3.0 * 0.044715 * x * x)


def gated(X, W_in, W_out, act):
    """(Y, G, U) of rows X [N, d]: Y = (act(G) * U) W_out, [G | U] = X W_in."""
    f = W_out.shape[0]
    Z = np.asarray(X, np.float64) @ np.asarray(W_in, np.float64)
    G, U = Z[:, :f], Z[:, f:]
    return (activation(G, act)[0] * U) @ np.asarray(W_out, np.float64), G, U


def gated_grad(dY, X, G, U, W_in, W_out, act):
    """(dX, dW_in, dW_out, dZ, H) at the projections G and U, with X for dW_in."""
    dY = np.asarray(dY, np.float64)
    a, slope = activation(G, act)
    dH = dY @ np.asarray(W_out, np.float64).T
    dZ = np.concatenate([dH * U * slope, dH * a], axis=1)
    H = a * U
    return (dZ @ np.asarray(W_in, np.float64).T, np.asarray(X, np.float64).T @ dZ, H.T @ dY, dZ, H)
