"""GPU: exponentials of the log probabilities, whose error does not grow with their
argument and does not add up over many rows; the example's reference with them.

Tolerances. The hardware's 2^p is right to one step (two half steps of U32), the factor
1 + c adds half a step of rounding and less than half a step by leaving out c^2 / 2 (c is
at most |p| half steps, 64 * 2^-24 here), and the product by the gradient of a row half a step
more: six half steps, whatever the argument is. Arguments z - lse are exact in these tests:
multiples of 1/16 below 128.

Sums over many rows: log probabilities of -8 to -16 are rounded to fp32 by up to 2^-21, evenly
spread, so by 2^-21 / sqrt(3) in the root mean square; a row's own fp32 additions stay below
U32 * sqrt(n) for n = vocab / 256 terms of a thread, and are independent from row to row. N rows together
are off by six times sqrt(N) times that, but for what is the same in every row: each
exponential's two half steps at most, taken as evenly spread over their two signs."""

import math
import os
import sys

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from train_helpers import U32, assert_within, f64, half_step, normal

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("vocab", [600, 20001])
def test_probabilities_far_below_the_sum(vocab, entropy):
    """fp32 gradients of entries whose probabilities are down to exp(-80)."""
    require_gpu()
    rows = 3
    g = torch.Generator().manual_seed(vocab)
    logits = torch.randint(-64 * 16, 0, (rows, vocab), generator=g).float().cuda() / 16
    lse = torch.tensor([0.0, 5.0, 16.0], device="cuda")
    tokens = torch.tensor([0, vocab - 1, 17], device="cuda")
    dlogps = torch.tensor([1.0, -0.5, 2.0], device="cuda")
    H = torch.tensor([3.0, 2.5, 1.0], device="cuda")
    dentropy = torch.tensor([0.25, 0.5, -1.0], device="cuda") if entropy else None
    got = nsmi.ns_token_logps_grad(logits, tokens, lse, H, dlogps, dentropy)
    x = f64(logits) - f64(lse)[:, None]
    p, k = np.exp(x), f64(dlogps)[:, None] * np.ones_like(x)
    bound = 6 * U32 * p * np.abs(k)
    if entropy:   # h (x + H) + g: two roundings of sums of magnitudes up to these
        size = np.abs(f64(dentropy)[:, None]) * (np.abs(x) + f64(H)[:, None]) + np.abs(k)
        k = k + f64(dentropy)[:, None] * (x + f64(H)[:, None])
        bound = (6 + 3) * U32 * p * size
    want = -p * k
    want[np.arange(rows), tokens.cpu()] += f64(dlogps)
    assert_within(got, want, bound + half_step(want, SF), "dlogits")


def test_sums_of_many_rows_agree_with_the_preference_loss():
    """The same logits by both operators: log probabilities of 8000 positions."""
    require_gpu()
    vocab, length = 32000, 4000
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn((2, length, vocab), generator=gen, device="cuda").mul_(2.5).to(BF)
    labels = torch.randint(0, vocab, (2, length), generator=gen, device="cuda")
    sums = nsmi.ns_preference_loss(logits, labels, torch.zeros(2, device="cuda"))[2]
    logps = nsmi.ns_token_logps(logits, labels)[0].double().sum(-1)
    row = 2.0 ** -20 / math.sqrt(3) + U32 * math.sqrt(vocab / 256)   # (down to -32: half a step is 2^-20)
    each = 6 * math.sqrt(length) * row + U32 * 1e5                   # (the sums themselves are rounded to fp32)
    off = (logps - sums.double()).cpu().numpy()
    assert np.all(np.abs(off) < each), (off, each)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_log_sums_are_off_to_both_sides(dtype):
    """The mean over many rows of what lse is off by: what is the same in every row."""
    require_gpu()
    rows, vocab = 2000, 128000
    gen = torch.Generator(device="cuda").manual_seed(2)
    off = []
    for _ in range(2):
        logits = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(2.5).to(dtype)
        tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")
        lse = nsmi.ns_token_logps(logits, tokens)[1].double()
        for a in range(0, rows, 200):
            off.append(lse[a:a + 200] - torch.logsumexp(logits[a:a + 200].double(), -1))
    off = torch.cat(off).cpu().numpy()
    row = 2.0 ** -21 / math.sqrt(3) + U32 * math.sqrt(vocab / 256) / 16   # (256 threads' sums, independent)
    assert abs(off.mean()) < 6 * row / math.sqrt(len(off)) + 0.2 * U32, (off.mean() / U32, off.std() / U32)


def test_reference_of_the_example_adds_up_like_the_policy():
    """Its reference is the policy as it starts, so that the first step's margins are 0 but for
    the roundings of a sequence's log probability (half a step) and of its positions (32 of them)."""
    require_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import preference_training as P
    given = []

    def loss(logits, labels, ref_logps, **kw):
        given.append((logits.clone(), labels, ref_logps))
        return real(logits, labels, ref_logps, **kw)

    real, nsmi.ns_preference_loss = nsmi.ns_preference_loss, loss
    try:
        P.train(steps=1)
    finally:
        nsmi.ns_preference_loss = real
    logits, labels, ref = given[0]
    assert ref.dtype == torch.float32
    tokens = nsmi.ns_token_logps(logits, labels)[0].double().cpu().numpy()
    assert np.array_equal(ref.cpu().numpy(), tokens.sum(-1).astype(np.float32))


@pytest.mark.parametrize("rows, vocab", [(4096, 65536), (4096, 16384), (600, 65536)])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_small_entries_are_not_lost_beside_long_sums(rows, vocab, dtype):
    """Rows whose small entries are many and far below the largest: a thread's sum of a
    thousand of them in fp32 drops what lies below half a step of it, always to one side. Sums of
    64 terms in fp32 lose 1 half step so at this spread, of 256 5, of 1024 20 (a model of the
    additions on the CPU, 65536 entries); those of 64 are allowed for, three times."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((rows, vocab), generator=gen, device="cuda").mul_(4.0).to(dtype)
    lse = nsmi.ns_token_logps(logits, torch.zeros(rows, dtype=torch.int64, device="cuda"), top=5)[1].double()
    off = torch.cat([lse[a:a + 256] - torch.logsumexp(logits[a:a + 256].double(), -1) for a in range(0, rows, 256)])
    off = off.cpu().numpy()
    row = 2.0 ** -20 / math.sqrt(3)   # lse of 16 to 32
    assert abs(off.mean()) < 6 * row / math.sqrt(rows) + 3 * U32, (off.mean() / U32, off.std() / U32)
