"""The float64 reference of the token operators, pinned on its own: gradients
against central differences, cross entropy and distillation against values
worked out by other means, and rows that take no part."""
import math

import numpy as np
import pytest

from oracle import tokens as ot


def _case(seed, N=5, d=6, V=11, k=3):
    r = np.random.default_rng(seed)
    X, E = r.standard_normal((N, d)), r.standard_normal((V, d))
    ids = np.stack([r.permutation(V)[:k] for _ in range(N)])
    t = r.standard_normal((N, k))
    g = r.standard_normal(N)
    return X, E, ids, t, g


def test_uniform_logits_give_log_V():
    X, E = np.zeros((2, 4)), np.ones((7, 4))
    loss, lse, _, _ = ot.target_loss(X, E, np.array([[3], [0]]), np.ones((2, 1)))
    np.testing.assert_allclose(loss, math.log(7))
    np.testing.assert_allclose(lse, math.log(7))


def test_teacher_equal_to_student_gives_zero_loss_and_gradient():
    """k = V and the teacher's logits are the student's: KL = 0."""
    X, E, _, _, g = _case(1)
    ids = np.tile(np.arange(11), (5, 1))
    z = 0.7 * X @ E.T
    for tau in (0.5, 1.0, 3.0):
        q = ot.teacher_weights(ids, z, 11, tau)
        loss, _, dX, dE = ot.target_loss(X, E, ids, q, 0.7, tau, g)
        np.testing.assert_allclose(loss, 0.0, atol=1e-12)
        np.testing.assert_allclose(dX, 0.0, atol=1e-12)
        np.testing.assert_allclose(dE, 0.0, atol=1e-12)


@pytest.mark.parametrize("scale,tau", [(1.0, 1.0), (0.5, 2.0), (1.5, 0.7)])
def test_gradients_match_central_differences(scale, tau):
    X, E, ids, t, g = _case(2)
    ids[1] = -1                               # a row without target
    ids[2, 1] = ids[2, 0]                     # one id named twice
    q = ot.teacher_weights(ids, t, 11, tau)

    def total(X, E):
        return float(np.sum(g * ot.target_loss(X, E, ids, q, scale, tau)[0]))

    _, _, dX, dE = ot.target_loss(X, E, ids, q, scale, tau, g)
    h = 1e-6
    for A, dA in ((X, dX), (E, dE)):
        for at in np.ndindex(*A.shape):
            keep = A[at]
            A[at] = keep + h
            up = total(X, E)
            A[at] = keep - h
            down = total(X, E)
            A[at] = keep
            assert abs((up - down) / (2 * h) - dA[at]) < 1e-7
    assert not dX[1].any()


def test_embedding_gradient_is_the_adjoint_of_the_lookup():
    """<dY, embed(E)> = <embed_grad(dY), E>, and the per-sample norms are
    those of each sample's own gradient."""
    r = np.random.default_rng(3)
    ids = r.integers(-1, 5, (4, 9))
    ids[3] = -1
    E, dY = r.standard_normal((5, 3)), r.standard_normal((4, 9, 3))
    dE = ot.embed_grad(ids, dY, 5, 2.5)
    assert abs(np.sum(dY * ot.embed(ids, E, 2.5)) - np.sum(dE * E)) < 1e-12
    n2 = ot.embed_norms_sq(ids, dY, 5, 2.5)
    assert n2[3] == 0.0
    one = np.zeros((5, 3))
    for t in range(9):
        if ids[0, t] >= 0:
            one[ids[0, t]] += 2.5 * dY[0, t]
    assert abs(n2[0] - np.sum(one ** 2)) < 1e-12


def test_teacher_weights_of_masked_entries():
    ids = np.array([[2, -1, 4], [-1, -1, -1], [1, 2, 3], [0, 1, 9]])
    t = np.array([[0.0, 9.0, 0.0], [1.0, 1.0, 1.0], [-np.inf] * 3, [1.0, -np.inf, 5.0]])
    q = ot.teacher_weights(ids, t, 5, 1.0)
    np.testing.assert_allclose(q, [[0.5, 0, 0.5], [0, 0, 0], [0, 0, 0], [1, 0, 0]])
