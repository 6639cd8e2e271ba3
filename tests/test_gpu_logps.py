"""GPU: log probabilities of given tokens with entropy and likeliest entries, and
their gradient, against the fp64 oracle.

Tolerances. x = z - m is rounded once, its exponential's argument once more: a term
is off by (2 |x| + 4) half steps, relative. A thread adds its terms in fp32, 64 or so
a step of 16384 (4096 in short rows), then everything is 64 bits: at most
vocab / 64 + 64 half steps. lse, entropy and log probabilities follow from both
sums; each is rounded once to fp32."""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import heads_oracle as H
from train_helpers import U32, assert_within, f64, half_step, normal, strided_rows, untouched

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def make(seed, rows, vocab, dtype, scale=3.0, ids=torch.int64, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    tokens[torch.rand(rows, generator=g) < ignored] = -100
    return normal(seed, (rows, vocab), dtype, scale), tokens.to(ids).cuda()


def sums_error(z, lse, vocab):
    """How far log(sum exp x) and sum x exp x / sum exp x may be off, each row."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        x = z - z.max(-1, keepdims=True)
        p = np.exp(z - lse[:, None])
        size = np.nansum(np.where(p > 0, p * np.abs(x), 0.0), -1)
        second = np.nansum(np.where(p > 0, p * x * x, 0.0), -1)
    chain = vocab / 64 + 64
    return (2 * size + 4 + chain) * U32, (2 * second + (8 + 2 * chain) * (size + 1)) * U32


def check(logits, tokens, top, **kw):
    got = nsmi.ns_token_logps(logits, tokens, top=top, **kw)
    z = f64(logits)
    want = H.token_logps(z, tokens.cpu().numpy(), top)
    e_lse, e_h = sums_error(z, want[1], z.shape[1])
    logps, lse, entropy, top_logps, top_ids = got
    assert_within(logps, want[0], e_lse + half_step(want[0], SF), "logps")
    assert_within(lse, want[1], e_lse + half_step(want[1], SF), "lse")
    assert_within(entropy, want[2], e_lse + e_h + half_step(want[2], SF), "entropy")
    if top:
        assert top_ids.dtype == tokens.dtype
        assert np.array_equal(top_ids.cpu().numpy(), want[4])
        assert_within(top_logps, want[3], e_lse[:, None] + half_step(want[3], SF), "top")
    else:
        assert top_logps is None and top_ids is None
    return got


SIZES = [(1, 1), (3, 2), (5, 7), (4, 8), (7, 100), (2, 511), (3, 513), (9, 1001), (5, 2048), (6, 2049), (3, 4097),
         (2, 16383), (2, 16385), (1, 50021), (1, 131072), (2500, 130)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_sizes(size, dtype):
    require_gpu()
    rows, vocab = size
    for top in sorted({0, 1, min(5, vocab), min(20, vocab), min(64, vocab)}):
        check(*make(rows + vocab, rows, vocab, dtype, ids=torch.int32 if top == 5 else torch.int64), top)


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("vocab", [300, 5000, 40000])
def test_orders_that_are_hard_to_choose_from(dtype, vocab):
    """Rising and falling rows, ties everywhere, few values, signed zeros."""
    require_gpu()
    ramp = torch.linspace(-8, 8, vocab, device="cuda")
    tokens = torch.arange(6, device="cuda") * 3
    rows = torch.stack([ramp, ramp.flip(0), torch.zeros_like(ramp), torch.full_like(ramp, 2.5),
                        torch.where(torch.arange(vocab, device="cuda") % 2 == 0, 0.0, -0.0),
                        (torch.arange(vocab, device="cuda") * 7919 % 5).float()]).to(dtype)
    for top in (1, 20, 64):
        check(rows, tokens, top)


def test_masked_entries():
    """-inf and the type's lowest value where a mask stands; rows with little left."""
    require_gpu()
    for dtype in (BF, HF, SF):
        low = torch.finfo(dtype).min
        for vocab in (90, 20000):
            logits, tokens = make(5, 6, vocab, dtype, ignored=0)
            tokens[:] = 3
            logits[0, 10:] = float("-inf")
            logits[1, ::2] = float("-inf")
            logits[2, 4:] = low
            logits[3] = float("-inf")
            logits[3, 3] = 1.0
            logits[4] = low
            logits[5, 3] = float("-inf")
            check(logits, tokens, 20)
    logits = torch.full((2, 300), float("-inf"), device="cuda")
    logps, lse, entropy, top_logps, ids = nsmi.ns_token_logps(logits, tokens[:2], top=4)
    assert torch.isnan(logps).all() and torch.isnan(entropy).all() and (lse == float("-inf")).all()
    assert ids.tolist() == [[0, 1, 2, 3]] * 2


@pytest.mark.parametrize("vocab", [70, 30000])
def test_nan_and_infinite_logits(vocab):
    require_gpu()
    logits, tokens = make(6, 5, vocab, SF, ignored=0)
    clean = nsmi.ns_token_logps(logits, tokens, top=5)
    logits[1, 7] = float("nan")
    logits[3, 9] = float("inf")
    logits[4] = float("nan")
    logits[4, 50] = 1.0
    got = nsmi.ns_token_logps(logits, tokens, top=5)
    for a, b in zip(got[:4], clean[:4]):
        assert torch.isnan(a[[1, 4]]).all() and torch.isnan(a[3]).all()
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert torch.equal(got[4][[0, 2]], clean[4][[0, 2]])
    z = torch.nan_to_num(logits[1], nan=-1e30)
    assert got[4][1].tolist() == torch.sort(z, descending=True, stable=True).indices[:5].tolist()
    assert got[4][3, 0] == 9 and got[4][4].tolist() == [50, -1, -1, -1, -1]


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("top", [5, 32, 33, 64])
def test_likeliest_beside_many_nan(dtype, top):
    """Whole vectors of NaN, and single ones, between entries that rise, fall or lie anywhere."""
    require_gpu()
    for vocab in (130, 3000, 50021):
        z, tokens = make(13, 6, vocab, dtype, ignored=0)
        z[1] = torch.linspace(-8, 8, vocab, device="cuda").to(dtype)
        z[2] = z[1].flip(0)
        at = torch.arange(vocab, device="cuda")
        z[:3, at // 8 % 2 == 1] = float("nan")
        z[3, at // 64 % 3 != 1] = float("nan")
        z[4, at % 2 == 0] = float("nan")
        z[5, 60:] = float("nan")
        ids = nsmi.ns_token_logps(z, tokens, top=top)[4]
        order = torch.sort(torch.nan_to_num(z.float(), nan=-1e30), dim=-1, descending=True, stable=True).indices
        left = (~z.isnan()).sum(-1, keepdim=True)
        want = torch.where(torch.arange(top, device="cuda") < left, order[:, :top], -1)
        assert torch.equal(ids, want)


def test_layouts():
    """Rows further apart, odd addresses, more dimensions, int32 tokens, strided tokens."""
    require_gpu()
    logits, tokens = make(7, 12, 1003, BF)
    want = check(logits, tokens, 4)
    view, store = strided_rows(logits, 5, 3)
    got = check(view, tokens, 4)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and untouched(store, view)
    got = nsmi.ns_token_logps(logits.view(3, 4, 1003), tokens.view(3, 4), top=4)
    assert got[0].shape == (3, 4) and got[4].shape == (3, 4, 4)
    assert all(torch.equal(a.flatten(), b.flatten()) for a, b in zip(got, want))
    got = nsmi.ns_token_logps(logits, tokens.repeat_interleave(2)[::2], top=4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    none = nsmi.ns_token_logps(logits[:0], tokens[:0], top=4)
    assert none[0].shape == (0,) and none[4].shape == (0, 4)
    one = nsmi.ns_token_logps(logits[0], torch.tensor(5, device="cuda"))
    assert one[0].shape == ()


def test_slices_of_sequences():
    """All positions but the last of each sequence, as a shifted loss takes them; the gradient in place and not."""
    require_gpu()
    for vocab in (203, 5000, 40000):
        whole, _ = make(12, 3 * 5, vocab, BF)
        whole = whole.view(3, 5, vocab).clone()
        tokens = torch.randint(-30, vocab, (3, 4)).cuda()
        part = whole[:, :-1]
        want = nsmi.ns_token_logps(part.contiguous(), tokens, top=3)
        got = nsmi.ns_token_logps(part, tokens, top=3)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        dl, dh = normal(1, (3, 4)), normal(2, (3, 4))
        args = (tokens, got[1], got[2], dl)
        d = nsmi.ns_token_logps_grad(part.contiguous(), *args, dentropy=dh)
        assert torch.equal(nsmi.ns_token_logps_grad(part, *args, dentropy=dh), d)
        last = whole[:, -1].clone()
        back = nsmi.ns_token_logps_grad(part, *args, dentropy=dh, out=part)
        assert back.data_ptr() == whole.data_ptr() and torch.equal(part, d) and torch.equal(whole[:, -1], last)
        with pytest.raises(ValueError):
            nsmi.ns_token_logps_grad(part, *args, out=whole[:, :-1].as_strided((3, 4, vocab), (4 * vocab, vocab, 1)))
        with pytest.raises(ValueError):
            nsmi.ns_token_logps(whole.transpose(0, 1)[:4], tokens.t())


def test_a_row_does_not_depend_on_the_others():
    """Few rows are cut into pieces, many are not: the same likeliest entries, sums within their errors."""
    require_gpu()
    logits, tokens = make(8, 2100, 20000, BF, ignored=0)
    many = check(logits[:], tokens, 20)
    few = check(logits[:3], tokens[:3], 20)
    assert torch.equal(many[4][:3], few[4])


def check_grad(logits, tokens, with_entropy, out=None, seed=3):
    rows, vocab = logits.shape
    _, lse, entropy, _, _ = nsmi.ns_token_logps(logits, tokens)
    dl = normal(seed, (rows,))
    dh = normal(seed + 1, (rows,)) if with_entropy else None
    z, l64, h64 = f64(logits), f64(lse), f64(entropy)
    got = nsmi.ns_token_logps_grad(logits, tokens, lse, entropy if with_entropy else None, dl, dh, out=out)
    dh64 = None if dh is None else f64(dh)
    want = H.token_logps_grad(z, tokens.cpu().numpy(), l64, h64, f64(dl), dh64)
    with np.errstate(invalid="ignore"):
        x = np.maximum(z - l64[:, None], -150.0)
    p = np.exp(x)
    slope = np.abs(f64(dl))[:, None] + (0 if dh is None else np.abs(dh64)[:, None] * (np.abs(x) + np.abs(h64)[:, None]))
    slack = (3 * np.abs(x) + 8) * U32 * p * slope + 4 * U32 * np.abs(want)
    slack += U32 * np.abs(f64(dl))[:, None]   # a sum with the token's own share
    assert got.dtype == logits.dtype
    assert_within(got, want, half_step(want, logits.dtype) + slack, "dlogits")
    return got


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_gradient(size, dtype):
    require_gpu()
    for with_entropy in (False, True):
        check_grad(*make(sum(size), *size, dtype), with_entropy)


def test_gradient_in_place_masked_and_strided():
    require_gpu()
    logits, tokens = make(9, 7, 3001, BF)
    logits[2, 100:] = float("-inf")
    logits[3, ::3] = torch.finfo(BF).min
    want = check_grad(logits, tokens, True)
    view, store = strided_rows(logits, 3, 1)
    got = check_grad(view, tokens, True, out=view)
    assert torch.equal(got, want) and untouched(store, view)
    out, outer = strided_rows(logits, 9, 5)
    assert torch.equal(check_grad(logits, tokens, True, out=out), want) and untouched(outer, out)


def test_gradient_of_one_part():
    """Either gradient may be left out; both parts add up."""
    require_gpu()
    logits, tokens = make(10, 6, 700, SF)
    _, lse, entropy, _, _ = nsmi.ns_token_logps(logits, tokens)
    dl, dh = normal(1, (6,)), normal(2, (6,))
    both = f64(nsmi.ns_token_logps_grad(logits, tokens, lse, entropy, dl, dh))
    a = f64(nsmi.ns_token_logps_grad(logits, tokens, lse, None, dl))
    b = f64(nsmi.ns_token_logps_grad(logits, tokens, lse, entropy, None, dh))
    scale = np.abs(a) + np.abs(b)
    assert (np.abs(a + b - both) <= 64 * U32 * scale + 1e-30).all()


def test_gradient_against_differences():
    """The entropy's gradient against differences of the call itself."""
    require_gpu()
    logits, tokens = make(11, 3, 50, SF, scale=1.0, ignored=0)
    _, lse, entropy, _, _ = nsmi.ns_token_logps(logits, tokens)
    ones = torch.ones(3, device="cuda")
    d = f64(nsmi.ns_token_logps_grad(logits, tokens, lse, entropy, ones, ones))
    step = 2.0 ** -5
    for v in range(0, 50, 7):
        up, down = logits.clone(), logits.clone()
        up[:, v] += step
        down[:, v] -= step
        up, down = nsmi.ns_token_logps(up, tokens), nsmi.ns_token_logps(down, tokens)
        diff = (f64(up[0]) + f64(up[2]) - f64(down[0]) - f64(down[2])) / (2 * step)
        # third derivatives of both are below 6 and 6 (3 + |log p|); values of about 8 are good to 2^-20
        assert np.abs(diff - d[:, v]).max() < step ** 2 / 6 * 60 + 2.0 ** -20 / step
