"""The fp64 forms of the operators around the matrix update: their gradients
against central differences of their own forward, and known values.

A central difference of step d in fp64 is off by O(d^2) of the third
derivative plus rounding O(2^-52 / d); with d = 1e-5 both are below 1e-9 for
values of order one.
"""

import numpy as np
import pytest

from oracle import train_oracle as O

D = 1e-5


def _slope(f, x, direction):
    return (f(x + D * direction) - f(x - D * direction)) / (2 * D)


def test_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(0)
    table, ids = rng.standard_normal((7, 5)), np.array([0, 3, 3, 6, -1, 9, 3])
    g = rng.standard_normal((7, 5))
    out = O.embedding(table, ids, 2.0)
    assert np.all(out[4] == 0) and np.all(out[5] == 0)
    grad, mag, n = O.embedding_grad(g, ids, 7, 2.0)
    assert n.tolist() == [1, 0, 0, 3, 0, 0, 1]
    # <dL/dtable, t> == <g, embedding(t)> for a linear map
    t = rng.standard_normal((7, 5))
    assert np.isclose(np.sum(grad * t), np.sum(g * O.embedding(t, ids, 2.0)), rtol=1e-13)
    padded, _, n = O.embedding_grad(g, ids, 7, 2.0, padding_idx=3)
    assert np.all(padded[3] == 0) and n[3] == 0


@pytest.mark.parametrize("with_dh", [False, True])
def test_rms_norm_gradient_against_differences(with_dh):
    rng = np.random.default_rng(1)
    h, w, dy = rng.standard_normal((3, 9)), rng.standard_normal(9), rng.standard_normal((3, 9))
    dh = rng.standard_normal((3, 9)) if with_dh else None
    dx, dw = O.rms_norm_grad(dy, h, w, 1e-3, dh)

    def loss_h(x):
        return np.sum(dy * O.rms_norm(x, w, 1e-3)[0]) + (np.sum(dh * x) if with_dh else 0.0)

    for _ in range(3):
        t = rng.standard_normal(h.shape)
        assert np.isclose(_slope(loss_h, h, t), np.sum(dx * t), rtol=1e-7, atol=1e-7)
        s = rng.standard_normal(9)
        slope = _slope(lambda x: np.sum(dy * O.rms_norm(h, x, 1e-3)[0]), w, s)
        assert np.isclose(slope, np.sum(dw * s), rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
def test_preference_gradient_against_differences(smoothing):
    rng = np.random.default_rng(2)
    z = rng.standard_normal((4, 5, 11))
    labels = rng.integers(0, 11, (4, 5))
    labels[0, :2] = -100
    labels[3] = -100                       # a sequence with nothing counted
    ref, dl = rng.standard_normal(4) - 10, rng.standard_normal(2)
    grad = O.preference_loss_grad(z, labels, ref, dl, 0.5, smoothing)
    assert np.all(grad[0, :2] == 0) and np.all(grad[3] == 0)
    for _ in range(3):
        t = rng.standard_normal(z.shape)
        slope = _slope(lambda x: np.sum(dl * O.preference_loss(x, labels, ref, 0.5, smoothing)[0]),
                       z, t)
        assert np.isclose(slope, np.sum(grad * t), rtol=1e-7, atol=1e-7)


def test_preference_loss_known_values():
    z = np.zeros((2, 1, 4))
    losses, margins, logps, lse = O.preference_loss(z, np.array([[1], [2]]), np.zeros(2), 0.3, 0.0)
    assert np.isclose(losses[0], np.log(2)) and margins[0] == 0
    assert np.allclose(logps, -np.log(4)) and np.allclose(lse, np.log(4))


def test_adamw_first_step_moves_by_lr():
    # from zero state, m / (1 - b1) = g and sqrt(v / (1 - b2)) = |g|
    w, m, v = O.adamw([1.0, -2.0], [0.3, -0.7], [0, 0], [0, 0], 1, 0.01, 0.9, 0.999, 0.0, 0.0)
    assert np.allclose(w, [0.99, -1.99]) and np.allclose(m, [0.03, -0.07])
    w, _, _ = O.adamw([1.0], [0.0], [0.0], [1.0], 5, 0.01, 0.9, 0.999, 1e-8, 0.5)
    assert np.allclose(w, 1 - 0.005)
