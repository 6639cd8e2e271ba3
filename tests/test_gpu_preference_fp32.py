"""The preference loss's gradient in fp32 as a function of what it is given:
margins, lse, dlosses and logits, taken as they are.

The differences z - lse are exact here (multiples of 2^-10 below 64), so an
element k ([v == label] - exp(z - lse)) carries only the kernel's own roundings.
The factor k is computed in 64 bits and rounded once to fp32.
"""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import train_oracle as O
from train_helpers import U32, assert_within, f64

pytestmark = pytest.mark.gpu

LSE = 16.0


def _slope(margins, smoothing):
    """smoothing sigmoid(m) - (1 - smoothing) sigmoid(-m), without its cancellation."""
    e = np.exp(-np.abs(margins))
    return np.where(margins >= 0, smoothing - (1 - smoothing) * e, smoothing * e - (1 - smoothing)) / (1 + e)


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 0.5, 1.0])
def test_the_factor_of_a_pair(smoothing):
    """At a label whose probability is 2e-16 the gradient is k itself: no more
    than its one rounding away, also where its two terms nearly cancel."""
    require_gpu()
    m = torch.tensor([0.0, 1e-6, -1e-6, 3e-4, -0.7, 2.1972246, 2.1972, -2.1972246, 40.0, -40.0, 1e3, -1e3,
                      float("inf"), float("-inf")])
    n = len(m)
    logits = torch.full((2 * n, 1, 40), LSE - 36.0, device="cuda")
    labels = torch.full((2 * n, 1), 7, dtype=torch.int64, device="cuda")
    lse, dl = torch.full((2 * n, 1), LSE, device="cuda"), torch.linspace(-2, 3, n).cuda()
    g = f64(nsmi.ns_preference_loss_grad(logits, labels, m.cuda(), lse, dl, beta=0.1,
                                         label_smoothing=smoothing))
    s = float(np.float32(smoothing))
    k = f64(dl) * float(np.float32(0.1)) * _slope(f64(m), s)
    want = np.concatenate([k, -k])
    # 1 - p rounds to 1; the smallest k are subnormal
    assert_within(g[:, 0, 7], want, 1.01 * U32 * np.abs(want) + 2.0 ** -149, "k")
    plain = f64(dl) * float(np.float32(0.1)) * (s * O.sigmoid(f64(m)) - (1 - s) * O.sigmoid(-f64(m)))
    assert np.allclose(k, plain, rtol=1e-7, atol=1e-15)      # the formula of the header


@pytest.mark.parametrize("vocab", [7, 1000, 20001])
def test_the_probabilities(vocab):
    """exp(z - lse): two roundings' worth from the hardware's power of two, one
    for the correction, one for the product with k, and k's own."""
    require_gpu()
    rng = np.random.default_rng(vocab)
    z = (LSE + rng.integers(-36 * 1024, 1, (2, 3, vocab)) / 1024).astype(np.float32)
    z[:, 1, 0], z[0, 2, -1], z[1, 2, -1] = -np.inf, np.finfo(np.float32).min, LSE - 200
    labels = torch.tensor([[1, 2, -100], [0, -100, vocab - 1]]).cuda()
    margins, dl = torch.tensor([0.3]).cuda(), torch.tensor([1.7]).cuda()
    lse = torch.full((2, 3), LSE, device="cuda")
    g = f64(nsmi.ns_preference_loss_grad(torch.from_numpy(z).cuda(), labels, margins, lse, dl, beta=0.1))
    k = f64(dl) * float(np.float32(0.1)) * _slope(f64(margins), 0.0)
    k = np.concatenate([k, -k])[:, None, None]
    keep = (labels >= 0).cpu().numpy()[..., None]
    at = np.zeros(z.shape)
    np.put_along_axis(at, labels.clamp(min=0).cpu().numpy()[..., None], 1.0, -1)
    p = np.exp(z.astype(np.float64) - LSE)
    want = np.where(keep, k * (at - p), 0.0)
    # at a label, p's error counts and 1 - p and the product round
    slack = np.abs(k) * np.where(at > 0, 3 * p + 3 * (1 - p), 5 * p) * U32 * 1.01 + 2.0 ** -126
    assert_within(g, want, np.where(keep, slack, 0.0), "gradient")
