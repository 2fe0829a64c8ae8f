"""Float64 reference of the token operators at the two ends of a language
model: embedding lookup with its per-sample norms and gradient, softmax cross
entropy against a table, and distillation from a teacher's top k logits.

Written from the formulas, row by row and token by token, with whole logit
rows; no code is shared with the GPU path. An id outside [0, V) marks a
position that takes no part.
"""
from __future__ import annotations

import numpy as np

__all__ = [
    "embed", "embed_grad", "embed_norms_sq", "teacher_weights", "target_loss",
]


def embed(ids, E, scale=1.0):
    """Y[n] = scale * E[ids[n]], zero where the id lies outside [0, V)."""
    ids = np.asarray(ids)
    E = np.asarray(E, np.float64)
    Y = np.zeros((*ids.shape, E.shape[1]))
    for at in np.ndindex(*ids.shape):
        if 0 <= ids[at] < E.shape[0]:
            Y[at] = scale * E[ids[at]]
    return Y


def embed_grad(ids, dY, V, scale=1.0, sample_scales=None):
    """dE[v] = scale sum_i s_i sum_{t: ids[i, t] = v} dY[i, t]."""
    ids = np.asarray(ids)
    dY = np.asarray(dY, np.float64)
    dE = np.zeros((V, dY.shape[2]))
    for i in range(ids.shape[0]):
        s = 1.0 if sample_scales is None else float(sample_scales[i])
        for t in range(ids.shape[1]):
            if 0 <= ids[i, t] < V:
                dE[ids[i, t]] += scale * s * dY[i, t]
    return dE


def embed_norms_sq(ids, dY, V, scale=1.0):
    """||gradient of the table of sample i alone||_F^2 for every i."""
    return np.array([np.sum(embed_grad(ids[i:i + 1], dY[i:i + 1], V, scale) ** 2)
                     for i in range(np.asarray(ids).shape[0])])


def teacher_weights(top_ids, top_logits, V, tau):
    """q_j = softmax of t_j / tau over the entries whose id lies in [0, V);
    all zero when no such entry has a logit above -inf."""
    top_ids = np.asarray(top_ids)
    t = np.asarray(top_logits, np.float64) / tau
    q = np.zeros(t.shape)
    for at in np.ndindex(*t.shape[:-1]):
        ok = (top_ids[at] >= 0) & (top_ids[at] < V) & (t[at] > -np.inf)
        if ok.any():
            w = np.exp(t[at][ok] - t[at][ok].max())
            q[at][ok] = w / w.sum()
    return q


def target_loss(X, E, ids, q, scale=1.0, tau=1.0, dloss=None):
    """Loss against the target distribution that puts q_nj on ids_nj:
        loss_n = tau^2 sum_j q_nj (ln q_nj - ln p_n,id(j)),
        p_n = softmax_v(scale x_n . e_v / tau),
    its lse_n = ln sum_v exp(scale x_n . e_v / tau), and with dloss the
    gradients of sum_n dloss_n loss_n. Rows without weight give zeros.
    Returns (loss, lse, dX, dE), the last two None without dloss."""
    X = np.asarray(X, np.float64)
    E = np.asarray(E, np.float64)
    d, V = X.shape[-1], E.shape[0]
    rows = X.reshape(-1, d)
    ids = np.asarray(ids).reshape(rows.shape[0], -1)
    q = np.asarray(q, np.float64).reshape(rows.shape[0], -1)
    loss, lse = np.zeros(rows.shape[0]), np.zeros(rows.shape[0])
    dX, dE = np.zeros(rows.shape), np.zeros(E.shape)
    g = None if dloss is None else np.asarray(dloss, np.float64).reshape(-1)
    for n in range(rows.shape[0]):
        on = (q[n] > 0) & (ids[n] >= 0) & (ids[n] < V)
        if not on.any():
            continue
        z = E @ rows[n] * (scale / tau)
        m = z.max()
        lse[n] = m + np.log(np.sum(np.exp(z - m)))
        w, at = q[n][on], ids[n][on]
        loss[n] = tau ** 2 * np.sum(w * (np.log(w) - (z[at] - lse[n])))
        if g is not None:
            D = np.exp(z - lse[n]) * w.sum()
            np.subtract.at(D, at, w)
            D *= scale * tau * g[n]
            dX[n] = D @ E
            dE += np.outer(D, rows[n])
    lead = X.shape[:-1]
    if g is None:
        return loss.reshape(lead), lse.reshape(lead), None, None
    return loss.reshape(lead), lse.reshape(lead), dX.reshape(X.shape), dE
