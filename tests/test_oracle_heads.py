"""The oracle's gradients of the operators on heads and of the token log
probabilities against central differences of its own forward forms, and a few
closed forms."""

import numpy as np
import pytest

from oracle import heads_oracle as H


def differences(f, x, dout, step=1e-6):
    """Gradient of sum(f(x) * dout) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = np.sum(f(x) * dout)
        x[i] = keep - step
        down = np.sum(f(x) * dout)
        x[i] = keep
        g[i] = (up - down) / (2 * step)
    return g


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_qk_norm_rope_grad(interleaved, weighted):
    r = np.random.default_rng(1)
    x, dy, w = r.normal(size=(3, 2, 12)), r.normal(size=(3, 2, 12)), r.normal(size=12)
    angle = H.angles(r.integers(0, 50, (3, 3)), 1.0 / 10 ** np.arange(4), [2, 1, 1])
    w = w if weighted else None
    dx, dw = H.qk_norm_rope_grad(dy, x, w, angle, 1e-6, interleaved)
    want = differences(lambda x: H.qk_norm_rope(x, w, angle, 1e-6, interleaved), x, dy)
    assert np.abs(dx - want).max() < 1e-8
    if weighted:
        want = differences(lambda w: H.qk_norm_rope(x, w, angle, 1e-6, interleaved), w, dy)
        assert np.abs(dw - want).max() < 1e-8


def test_rotation_keeps_distances_between_positions():
    r = np.random.default_rng(2)
    q, k, freq = r.normal(size=8), r.normal(size=8), 0.3 ** np.arange(4)
    dots = []
    for shift in (0, 5, 100):
        a = H.rotate(np.stack([q, k])[:, None], H.angles(np.array([7, 3]) + shift, freq))[:, 0]
        dots.append(a[0] @ a[1])
    assert np.ptp(dots) < 1e-12 and abs(dots[0] - q @ k) > 1e-3


def test_attention_grad():
    r = np.random.default_rng(3)
    q, k, v = r.normal(size=(7, 4, 6)), r.normal(size=(7, 2, 6)), r.normal(size=(7, 2, 6))
    dout, ends = r.normal(size=(7, 4, 6)), [0, 1, 1, 5, 6]
    dout[6:] = 0
    out, lse, _ = H.attention(q, k, v, ends, 0.4)
    (dq, dk, dv), _ = H.attention_grad(dout, q, k, v, out, lse, ends, 0.4)
    f = lambda q, k, v: H.attention(q, k, v, ends, 0.4)[0]   # noqa: E731
    assert np.abs(dq - differences(lambda x: f(x, k, v), q, dout)).max() < 1e-8
    assert np.abs(dk - differences(lambda x: f(q, x, v), k, dout)).max() < 1e-8
    assert np.abs(dv - differences(lambda x: f(q, k, x), v, dout)).max() < 1e-8
    assert not dq[6].any() and not out[6].any()
    assert np.allclose(out[0], np.repeat(v[0], 2, axis=0))   # a row that sees itself alone


def test_token_logps_grad():
    r = np.random.default_rng(4)
    z, tokens = r.normal(size=(4, 9)), np.array([3, -100, 0, 9])
    z[2, 4] = -np.inf
    logps, lse, entropy, top_logps, ids = H.token_logps(z, tokens, 3)
    assert logps[1] == lse[3] == entropy[1] == 0 and (ids[[1, 3]] == -1).all()
    assert (ids[0] == np.argsort(-z[0])[:3]).all()
    dl, dh = r.normal(size=4), r.normal(size=4)
    d = H.token_logps_grad(z, tokens, lse, entropy, dl, dh)
    finite = z.copy()
    finite[2, 4] = -800.0
    want = differences(lambda z: H.token_logps(z, tokens)[0] * dl + H.token_logps(z, tokens)[2] * dh, finite,
                       np.ones(4))
    assert np.abs(d - want).max() < 1e-8 and d[2, 4] == 0


def test_ties_go_to_the_lowest_index():
    z = np.array([[1.0, 2.0, -0.0, 2.0, 0.0, np.nan, 1.0]])
    assert H.token_logps(z, [0], 7)[4].tolist() == [[1, 3, 0, 6, 2, 4, 5]]
