"""Preference loss and its gradient against the fp64 forms.

Tolerances. A term exp(z - max) carries the rounding of the product with
log2(e), at most |z - max| + 4 half steps, relative, and vanishes where
|z - max| is large: the sum over a row is off by fewer than A = R + 160 half
steps, with R the largest |z - max| that counts (terms below exp(-R) of the
largest do not matter: R = 20) and 160 for the additions of a thread, its
wave, its workgroup and the pieces. So lse is off by A half steps (absolute,
before its own rounding), a sequence's log probability by A times its counted
positions, a margin by beta times both sequences' errors, a loss by its
margin's error (its slope is at most 1). Beyond that each result is rounded
once. A gradient element is k (1 - p) or -k p: p is off by A + |lse| half
steps (lse is stored in fp32), relative, k by that of the margin, relative,
and 12 half steps.
"""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import train_oracle as O
from train_helpers import U32, assert_within, f64, half_step, normal, strided_rows, untouched

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
A = 20 + 160


def _labels(seed, n, length, vocab, ignored=0.4):
    rng = np.random.default_rng(seed)
    labels = rng.integers(0, vocab, (n, length))
    labels[rng.random((n, length)) < ignored] = -100
    return labels


def _check(logits, labels, ref, beta, smoothing, dlosses=None, labels_dev=None, what=""):
    """Runs both calls, checks every output; returns them."""
    b32, s32 = float(np.float32(beta)), float(np.float32(smoothing))
    dev = torch.from_numpy(labels).cuda() if labels_dev is None else labels_dev
    out = nsmi.ns_preference_loss(logits, dev, ref, beta=beta, label_smoothing=smoothing)
    losses, margins, logps, lse = out
    z = f64(logits)
    wl, wm, wp, we = O.preference_loss(z, labels, f64(ref), b32, s32)
    pairs = len(wl)
    keep = (labels >= 0) & (labels < z.shape[2])
    n = keep.sum(-1)
    assert_within(lse, we, np.where(keep, (A + np.abs(we)) * U32, 0.0), what + " lse")
    logp_off = A * U32 * n
    assert_within(logps, wp, logp_off + 1.01 * U32 * np.abs(wp) + 1e-12, what + " logps")
    margin_off = abs(b32) * (logp_off[:pairs] + logp_off[pairs:]) + 1e-12
    assert_within(margins, wm, margin_off + 1.01 * U32 * np.abs(wm), what + " margins")
    assert_within(losses, wl, margin_off + 1.01 * U32 * (np.abs(wl) + margin_off), what + " losses")
    dl = normal(5, (pairs,)) if dlosses is None else dlosses
    grad = nsmi.ns_preference_loss_grad(logits, dev, margins, lse, dl, beta=beta,
                                        label_smoothing=smoothing)
    want = O.preference_loss_grad(z, labels, f64(ref), f64(dl), b32, s32)
    sig = O.sigmoid(wm)
    k = np.abs(f64(dl) * b32) * (s32 * sig + (1 - s32) * (1 - sig))   # magnitudes: no cancellation
    k_off = k * (12 * U32 + 2 * margin_off + 4 * U32 * np.abs(wm))
    k, k_off = np.concatenate([k, k])[:, None, None], np.concatenate([k_off, k_off])[:, None, None]
    p = np.exp(z - we[..., None])
    at = np.zeros_like(z)
    np.put_along_axis(at, np.where(keep, labels, 0)[..., None], 1.0, -1)
    slack = k_off * np.abs(at - p) + (k + k_off) * (p * (A + np.abs(we[..., None])) + 2) * U32
    slack = np.where(keep[..., None], slack, 0.0) * 1.01
    assert grad.dtype == logits.dtype
    slack = slack + np.where(keep[..., None], 1.01 * half_step(np.abs(want) + slack, logits.dtype), 0.0)
    assert_within(grad, want, slack, what + " gradient")
    return losses, margins, logps, lse, grad


@pytest.mark.parametrize("pairs,length,vocab", [
    (1, 1, 1), (1, 1, 2), (2, 3, 7), (3, 5, 64), (1, 17, 1001), (2, 9, 8192), (1, 4, 8193), (1, 2, 50021),
    (5, 40, 777), (2, 1100, 130), (1, 3, 262147)])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_loss_and_gradient(pairs, length, vocab, dtype, smoothing):
    require_gpu()
    print("preference", pairs, length, vocab, dtype, smoothing, flush=True)
    logits = normal(vocab + length, (2 * pairs, length, vocab), dtype, 2.0)
    labels = _labels(vocab, 2 * pairs, length, vocab)
    n = ((labels >= 0).sum(-1) * -np.log(vocab + 1.0)).astype(np.float32)
    ref = torch.from_numpy(n).cuda()
    out = _check(logits, labels, ref, 0.1, smoothing)
    again = _check(logits, labels, ref, 0.1, smoothing,
                   labels_dev=torch.from_numpy(labels).to(torch.int32).cuda())
    assert all(torch.equal(x, y) for x, y in zip(out, again)), "int32 labels, or a second call"


def test_labels_outside_the_vocabulary_do_not_count():
    require_gpu()
    labels = np.array([[0, -100, 9, 2 ** 40], [-1, 10, 3, 3], [-100] * 4, [1, 2, 10 ** 9, 5]])
    logits = normal(1, (4, 4, 10), SF)
    logits[0, 1], logits[2], logits[3, 2] = float("nan"), float("inf"), float("nan")   # not counted
    out = nsmi.ns_preference_loss(logits, torch.from_numpy(labels).cuda(), torch.zeros(4, device="cuda"))
    clean = torch.nan_to_num(logits, nan=0.0, posinf=0.0)
    want = _check(clean, labels, torch.zeros(4, device="cuda"), 0.1, 0.0)
    assert all(torch.equal(x, y) for x, y in zip(out, want))
    g = nsmi.ns_preference_loss_grad(logits, torch.from_numpy(labels).cuda(), out[1], out[3],
                                     torch.ones(2, device="cuda"))
    assert torch.all(g[0, 1] == 0) and torch.all(g[2] == 0) and torch.all(g[3, 2] == 0)


def test_masked_entries_and_far_apart_logits():
    """-inf and the types' lowest value among the logits; logits of +-300."""
    require_gpu()
    for dtype in (BF, SF):
        logits = normal(2, (2, 6, 5000), dtype, 3.0)
        logits[:, :, 10:4000] = float("-inf")
        logits[:, 1, 4000:4500] = torch.finfo(dtype).min
        logits[:, 2] *= 100
        labels = np.array([[4999, 4600, 1, 2, 3, -100], [4, 5, 4700, 7, 8, 9]])
        _check(logits, labels, torch.zeros(2, device="cuda"), 0.01, 0.1)
        # pieces that hold nothing but masked entries
        wide = torch.full((2, 2, 40000), float("-inf"), dtype=dtype, device="cuda")
        wide[:, :, 39990:] = normal(3, (2, 2, 10), dtype)
        wide[1, 0, :5] = normal(4, (5,), dtype)
        _check(wide, np.array([[39991, 39999], [2, 39995]]), torch.zeros(2, device="cuda"), 0.5, 0.0)


def test_infinities_and_nan_follow_the_formula():
    require_gpu()
    logits = normal(3, (8, 2, 100), SF)
    labels = np.full((8, 2), 5)
    logits[0, 0, 5] = float("-inf")          # the preferred sequence is impossible: loss inf
    logits[5, 0, 5] = float("-inf")          # the other is: loss 0
    logits[2, 1, 7] = float("nan")
    logits[3, 0] = float("-inf")             # no entry left
    dev, ref = torch.from_numpy(labels).cuda(), torch.zeros(8, device="cuda")
    losses, margins, logps, lse = nsmi.ns_preference_loss(logits, dev, ref)
    assert torch.isinf(losses[0]) and losses[1] == 0
    assert margins[0] == float("-inf") and margins[1] == float("inf")
    assert torch.isnan(losses[2]) and torch.isnan(losses[3]) and torch.isnan(lse[2, 1])
    assert lse[3, 0] == float("-inf") and torch.isfinite(lse[2, 0])
    g = nsmi.ns_preference_loss_grad(logits, dev, margins, lse, torch.ones(4, device="cuda"))
    assert torch.isfinite(g[[0, 4, 1, 5]]).all() and torch.all(g[[1, 5]] == 0)
    assert g[0, 0, 5].item() == pytest.approx(-0.1, rel=1e-6)      # k (1 - 0)
    assert torch.isnan(g[2, 1]).any() and torch.isnan(g[3, 0]).all()
    # a smoothing of 0 or 1 leaves the other term out, infinite as it is
    l1 = nsmi.ns_preference_loss(logits, dev, ref, label_smoothing=1.0)[0]
    assert l1[0] == 0 and torch.isinf(l1[1])


def test_large_margins():
    require_gpu()
    logits = normal(4, (6, 3, 50), SF)
    labels = _labels(1, 6, 3, 50, 0.0)
    ref = torch.tensor([900.0, -900.0, 90.0, 0, 0, 0], device="cuda")
    for smoothing in (0.0, 0.2):
        _check(logits, labels, ref, 1.0, smoothing)


def test_empty_sequences_and_no_pairs():
    require_gpu()
    logits = torch.empty((4, 0, 9), device="cuda")
    labels = torch.empty((4, 0), dtype=torch.int64, device="cuda")
    ref = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    losses, margins, logps, lse = nsmi.ns_preference_loss(logits, labels, ref, beta=0.5)
    assert margins.tolist() == [1.0, 1.0] and logps.tolist() == [0.0] * 4 and lse.shape == (4, 0)
    assert losses.tolist() == pytest.approx([np.log1p(np.exp(-1.0))] * 2, rel=1e-6)
    g = nsmi.ns_preference_loss_grad(logits, labels, margins, lse, losses)
    assert g.shape == (4, 0, 9)
    none = nsmi.ns_preference_loss(logits[:0], labels[:0], ref[:0])
    assert [t.numel() for t in none] == [0, 0, 0, 0]


def test_strided_unaligned_and_in_place():
    require_gpu()
    for dtype in (BF, SF):
        full = normal(6, (4, 7, 1003), dtype)
        rows, _ = strided_rows(full, 5, 1)
        logits = rows.view(4, 7, 1003)
        labels = _labels(3, 4, 7, 1003)
        ref = torch.zeros(4, device="cuda")
        losses, margins, logps, lse, grad = _check(logits, labels, ref, 0.1, 0.1)
        same = _check(full, labels, ref, 0.1, 0.1)
        assert all(torch.equal(x, y) for x, y in zip((losses, margins, logps, lse, grad), same))
        dl, dev = normal(5, (2,)), torch.from_numpy(labels).cuda()
        view, store = strided_rows(torch.zeros(28, 1003, dtype=dtype, device="cuda"), 2, 3)
        nsmi.ns_preference_loss_grad(full, dev, margins, lse, dl, label_smoothing=0.1,
                                     out=view.view(4, 7, 1003))
        assert torch.equal(view.view(4, 7, 1003), grad) and untouched(store, view)
        inplace = nsmi.ns_preference_loss_grad(full, dev, margins, lse, dl, label_smoothing=0.1, out=full)
        assert inplace is full and torch.equal(full, grad)


def test_slices_of_positions_and_sequences():
    """logits[:, :-1], every second sequence, and labels[:, 1:] as they are."""
    require_gpu()
    for dtype, vocab in ((BF, 1003), (SF, 64)):
        full = normal(11, (8, 6, vocab), dtype)
        all_labels = torch.from_numpy(_labels(4, 8, 6, vocab)).cuda()
        ref, dl = normal(12, (4,)), normal(13, (2,))
        for pick in (lambda t: t[::2, :-1], lambda t: t[:4, 1:], lambda t: t[:4, 2:3], lambda t: t[4:]):
            logits, labels = pick(full), pick(all_labels)
            want = _check(logits.contiguous(), labels.cpu().numpy(), ref, 0.1, 0.1, dlosses=dl)
            out = nsmi.ns_preference_loss(logits, labels, ref, label_smoothing=0.1)
            assert all(torch.equal(a, b) for a, b in zip(out, want))
            g = nsmi.ns_preference_loss_grad(logits, labels, out[1], out[3], dl, label_smoothing=0.1)
            assert torch.equal(g, want[4])
            whole = full.clone()
            part = pick(whole)
            nsmi.ns_preference_loss_grad(part, labels, out[1], out[3], dl, label_smoothing=0.1, out=part)
            assert torch.equal(part, want[4])
            part.zero_()
            rest = full.clone()
            pick(rest).zero_()
            assert torch.equal(whole, rest)          # nothing beside the slice was written


def test_very_many_pairs():
    """More short sequences than a grid of large workgroups holds."""
    require_gpu()
    pairs = (1 << 22) - 1
    logits = torch.zeros((2 * pairs, 1, 3), dtype=BF, device="cuda")
    logits[5, 0, 1], logits[-1, 0, 2] = 2.0, 2.0
    labels = torch.ones((2 * pairs, 1), dtype=torch.int32, device="cuda")
    losses, margins, logps, lse = nsmi.ns_preference_loss(logits, labels, torch.zeros(2 * pairs, device="cuda"))
    up, down, flat = 2 - np.log(2 + np.exp(2.0)), -np.log(2 + np.exp(2.0)), -np.log(3.0)
    assert logps[5].item() == pytest.approx(up, rel=1e-6) and logps[-1].item() == pytest.approx(down, rel=1e-6)
    assert margins[5].item() == pytest.approx(0.1 * (up - flat), rel=1e-5)
    assert margins[-1].item() == pytest.approx(0.1 * (flat - down), rel=1e-5)
    assert losses[7].item() == pytest.approx(np.log(2.0), rel=1e-6)
    g = nsmi.ns_preference_loss_grad(logits, labels, margins, lse, torch.ones(pairs, device="cuda"))
    assert g[7, 0, 1].item() == pytest.approx(-0.05 * 2 / 3, rel=2 ** -8)
    assert g[pairs + 7, 0, 1].item() == pytest.approx(0.05 * 2 / 3, rel=2 ** -8)


def test_out_that_is_another_view_is_refused():
    require_gpu()
    full = normal(1, (2, 4, 24), SF)
    logits, labels = full[:, :-1], torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    out = nsmi.ns_preference_loss(logits, labels, torch.zeros(2, device="cuda"))
    other = full.view(-1)[:144].view(2, 3, 24)
    with pytest.raises(ValueError):
        nsmi.ns_preference_loss_grad(logits, labels, out[1], out[3], out[0], out=other)


def test_gradient_against_differences():
    """<gradient, t> against central differences of the fp64 forward."""
    require_gpu()
    logits, labels = normal(7, (6, 9, 83), SF), _labels(7, 6, 9, 83)
    ref, dl = normal(8, (6,)), normal(9, (3,))
    beta, d = 0.25, 1e-5
    out = nsmi.ns_preference_loss(logits, torch.from_numpy(labels).cuda(), ref, beta=beta)
    g = f64(nsmi.ns_preference_loss_grad(logits, torch.from_numpy(labels).cuda(), out[1], out[3], dl,
                                         beta=beta))
    z, t = f64(logits), f64(normal(10, (6, 9, 83)))
    f = lambda x: np.sum(f64(dl) * O.preference_loss(x, labels, f64(ref), beta, 0.0)[0])   # noqa: E731
    slope = (f(z + d * t) - f(z - d * t)) / (2 * d)
    assert abs(slope - np.sum(g * t)) <= 1e-6 + 2 * A * U32 * np.sum(np.abs(g * t))


def test_offsets_beyond_32_bits():
    require_gpu()
    pairs, length, vocab = 1, 9000, 150001
    logits = torch.zeros((2, length, vocab), dtype=BF, device="cuda")
    logits[1, -1, -1], logits[1, -2, 0] = 8.0, 8.0
    labels = torch.full((2, length), -100, dtype=torch.int64, device="cuda")
    labels[1, -1], labels[1, -2] = vocab - 1, 0
    losses, margins, logps, lse = nsmi.ns_preference_loss(logits, labels, torch.zeros(2, device="cuda"))
    one = 8 - np.log(vocab - 1 + np.exp(8.0))
    assert logps[0] == 0 and logps[1].item() == pytest.approx(2 * one, rel=1e-6)
    g = nsmi.ns_preference_loss_grad(logits, labels, margins, lse, torch.ones(1, device="cuda"),
                                     out=logits)
    assert torch.all(g[0] == 0) and torch.all(g[1, :-2] == 0)
    k = 0.1 / (1 + np.exp(margins.item()))
    assert g[1, -1, -1].item() == pytest.approx(k * (1 - np.exp(one)), rel=2 ** -8)
    assert g[1, -2, -1].item() == pytest.approx(-k * np.exp(-lse[1, -2].item()), rel=2 ** -8)
