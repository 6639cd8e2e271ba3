"""GPU: norm and rotation of queries and keys, and their gradient, against the
fp64 oracle.

Tolerances: an output is rounded once to its type (half a step); before that
each value carries fp32 errors. The sum of squares and the mean of a head's
products are sums of at most 256 terms over 4 to 64 lanes (at most 16 in a row on a
lane, 6 exchanges, a few operations behind: under 32 half steps), an angle is
rounded to 2^-26 turns (4e-7 of a value: 7 half steps) and its sine and cosine are
good to 2 half steps. In all less than 64 half steps of fp32 of the magnitudes
that enter."""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import heads_oracle as H
from train_helpers import U32, assert_within, f64, half_step, normal

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def freqs(pairs, theta=10000.0):
    return (theta ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float().cuda()


def make(seed, tokens, q_heads, k_heads, dim, rotary, dtype, axes=1, far=100000, ids=torch.int64):
    g = torch.Generator().manual_seed(seed)
    shape = (tokens,) if axes == 1 else (axes, tokens)
    positions = torch.randint(0, far, shape, generator=g).to(ids).cuda()
    return dict(q=normal(seed, (tokens, q_heads, dim), dtype), k=normal(seed + 1, (tokens, k_heads, dim), dtype, 3.0),
                q_weight=normal(seed + 2, (dim,), dtype), k_weight=normal(seed + 3, (dim,), dtype),
                positions=positions, inv_freq=freqs(rotary // 2))


def magnitude(x, interleaved, pairs):
    """|x_a| + |x_b| at both columns of each pair."""
    m = np.abs(x)
    a, b = H.pair_columns(pairs, interleaved)
    out = m.copy()
    out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


def check(c, sections=None, interleaved=False, weights=True, **outs):
    w = (c["q_weight"], c["k_weight"]) if weights else (None, None)
    got = nsmi.ns_qk_norm_rope(c["q"], c["k"], *w, c["positions"], c["inv_freq"], eps=EPS, sections=sections,
                               interleaved=interleaved, **outs)
    angle = H.angles(c["positions"].cpu().numpy(), f64(c["inv_freq"]), sections)
    for y, x, weight, name in ((got[0], c["q"], w[0], "q"), (got[1], c["k"], w[1], "k")):
        u = H.qk_norm_rope(f64(x), None if weight is None else f64(weight), angle * 0, EPS, interleaved)
        want = H.rotate(u, angle, interleaved)
        assert y.dtype == x.dtype
        assert_within(y, want, half_step(want, x.dtype) + 64 * U32 * magnitude(u, interleaved, angle.shape[1]), name)
    return got


SHAPES = [
    # tokens, q_heads, k_heads, dim, rotary
    (1, 1, 1, 4, 4), (3, 32, 8, 128, 128), (2, 5, 1, 128, 64), (7, 6, 2, 80, 80), (5, 4, 4, 256, 256),
    (4, 3, 3, 72, 32), (9, 2, 1, 20, 12), (6, 7, 1, 252, 252), (5, 1, 1, 96, 24), (3, 64, 1, 16, 16),
    (2100, 3, 1, 64, 64), (33, 2, 2, 32, 0), (17, 100, 3, 8, 8),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_forward(shape, dtype):
    require_gpu()
    check(make(sum(shape), *shape, dtype), interleaved=shape[0] % 2 == 0)


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_forward_kinds(dtype, interleaved, weights):
    require_gpu()
    check(make(3, 11, 6, 2, 128, 96, dtype, ids=torch.int32), interleaved=interleaved, weights=weights)
    check(make(4, 11, 6, 2, 64, 64, dtype, axes=3), sections=[16, 8, 8], interleaved=interleaved, weights=weights)
    check(make(5, 5, 2, 1, 72, 40, dtype, axes=4), sections=[0, 11, 0, 9], interleaved=interleaved, weights=weights)


def test_far_positions():
    """Positions where 32 bits would lose the angle; negative ones."""
    require_gpu()
    c = make(1, 64, 2, 1, 64, 64, SF, far=1 << 30)
    check(c)
    c["positions"] -= 1 << 29
    check(c)


def views(c, dtype):
    """q and k as parts of one projection's output."""
    t, hq, d = c["q"].shape
    hk = c["k"].shape[1]
    both = torch.full((t, hq + 2 * hk, d), float("nan"), dtype=dtype, device="cuda")
    both[:, :hq], both[:, hq:hq + hk] = c["q"], c["k"]
    return dict(c, q=both[:, :hq], k=both[:, hq:hq + hk]), both


@pytest.mark.parametrize("shape", [(9, 6, 2, 128, 128), (5, 3, 1, 72, 64)])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_parts_of_one_buffer_and_in_place(shape, dtype):
    require_gpu()
    c = make(2, *shape, dtype)
    want = check(c)
    v, both = views(c, dtype)
    got = check(v)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q, k = nsmi.ns_qk_norm_rope(v["q"], v["k"], v["q_weight"], v["k_weight"], v["positions"], v["inv_freq"],
                                eps=EPS, out_q=v["q"], out_k=v["k"])
    assert q.data_ptr() == both.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.isnan(both[:, shape[1] + shape[2]:].float()).all()   # the values are not touched


def test_heads_before_tokens_and_odd_addresses():
    require_gpu()
    c = make(6, 10, 4, 2, 64, 64, BF)
    want = check(c)
    flip = dict(c, q=c["q"].transpose(0, 1).contiguous().transpose(0, 1),
                k=c["k"].transpose(0, 1).contiguous().transpose(0, 1))
    assert flip["q"].stride(0) == 64
    out = torch.empty(4 * 10 * 64 + 3, dtype=BF, device="cuda")[3:].view(4, 10, 64).transpose(0, 1)
    got = check(flip, out_q=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    store = torch.empty(10 * 4 * 67 + 1, dtype=BF, device="cuda")[1:].view(10, 4, 67)[..., :64]
    store.copy_(c["q"])
    assert torch.equal(check(dict(c, q=store))[0], want[0])
    wide = dict(c, k=c["k"][:, :1].expand(10, 5, 64))       # one key head, read five times
    got = nsmi.ns_qk_norm_rope(wide["q"], wide["k"], c["q_weight"], c["k_weight"], c["positions"], c["inv_freq"])
    assert torch.equal(got[1], want[1][:, :1].expand(10, 5, 64))


def check_grad(c, sections=None, interleaved=False, weights=True, dw_dtype=None, seed=9, **outs):
    dtype, (t, hq, d), hk = c["q"].dtype, c["q"].shape, c["k"].shape[1]
    gq, gk = normal(seed, (t, hq, d), dtype, 0.1), normal(seed + 1, (t, hk, d), dtype, 0.1)
    if "on_dout" in outs:
        outs = dict(dq=gq, dk=gk)
    w = (c["q_weight"], c["k_weight"]) if weights else (None, None)
    g64 = (f64(gq), f64(gk))
    got = nsmi.ns_qk_norm_rope_grad(gq, gk, c["q"], c["k"], *w, c["positions"], c["inv_freq"], eps=EPS,
                                    sections=sections, interleaved=interleaved, dweight_dtype=dw_dtype, **outs)
    angle = H.angles(c["positions"].cpu().numpy(), f64(c["inv_freq"]), sections)
    for i, (x, weight) in enumerate(((c["q"], w[0]), (c["k"], w[1]))):
        w64 = None if weight is None else f64(weight)
        dx, dw = H.qk_norm_rope_grad(g64[i], f64(x), w64, angle, EPS, interleaved)
        mag = magnitude(g64[i], interleaved, angle.shape[1])
        if weight is None:
            assert got[2 + i] is None
            assert_within(got[i], dx, half_step(dx, dtype) + 64 * U32 * mag, f"dx {i}")
            continue
        n = f64(x)
        rstd = 1 / np.sqrt(np.mean(n * n, -1, keepdims=True) + EPS)
        n = np.abs(n * rstd)
        gw = mag * np.abs(w64)
        slack = 64 * U32 * rstd * (gw + n * np.mean(gw * n, -1, keepdims=True))
        assert_within(got[i], dx, half_step(dx, dtype) + slack, f"dx {i}")
        # a lane adds one term a round of heads and token, a workgroup eight lanes' and four waves'
        terms = -(-t // (4 * min(1024, -(-t // 4)))) * -(-(hq + hk) // 1) + 16
        out = got[2 + i]
        assert out.dtype == (dw_dtype or weight.dtype)
        assert_within(out, dw, half_step(dw, out.dtype) + (64 + terms) * U32 * np.sum(mag * n, (0, 1)), f"dw {i}")
    return got


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_gradient(shape, dtype):
    require_gpu()
    check_grad(make(sum(shape) + 7, *shape, dtype), interleaved=shape[0] % 2 == 1)


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_gradient_kinds(dtype, interleaved, weights):
    require_gpu()
    kw = dict(interleaved=interleaved, weights=weights)
    check_grad(make(13, 11, 6, 2, 128, 96, dtype), dw_dtype=SF if weights else None, **kw)
    check_grad(make(14, 4100, 3, 1, 64, 64, dtype, axes=3), sections=[16, 8, 8], **kw)
    check_grad(make(15, 5, 2, 1, 72, 40, dtype, axes=2), sections=[11, 9], on_dout=True, **kw)


def test_gradient_into_parts_of_one_buffer():
    require_gpu()
    c = make(21, 12, 6, 2, 128, 128, BF)
    want = check_grad(c)
    store = torch.full((12, 10, 128), float("nan"), dtype=BF, device="cuda")
    got = check_grad(c, dq=store[:, :6], dk=store[:, 6:8])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.isnan(store[:, 8:].float()).all()


def test_fp32_weights_and_no_tokens():
    require_gpu()
    c = make(22, 8, 4, 2, 64, 64, BF)
    c["q_weight"], c["k_weight"] = c["q_weight"].float(), c["k_weight"].float()
    check(c)
    check_grad(c)
    none = make(23, 0, 4, 2, 64, 64, BF)
    q, k = nsmi.ns_qk_norm_rope(none["q"], none["k"], none["q_weight"], none["k_weight"], none["positions"],
                                none["inv_freq"])
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    out = nsmi.ns_qk_norm_rope_grad(none["q"], none["k"], none["q"], none["k"], none["q_weight"],
                                    none["k_weight"], none["positions"], none["inv_freq"])
    assert not out[2].any() and not out[3].any()


def test_zero_rows_and_nan_rows():
    """A head of zeros stays zeros; a NaN stays in its own head."""
    require_gpu()
    c = make(24, 6, 3, 1, 64, 64, SF)
    c["q"][1, 2] = 0
    c["q"][4, 0, 5] = float("nan")
    q, k = nsmi.ns_qk_norm_rope(c["q"], c["k"], c["q_weight"], c["k_weight"], c["positions"], c["inv_freq"])
    assert not q[1, 2].any() and torch.isnan(q[4, 0]).all()
    q[4, 0] = 0
    assert torch.isfinite(q).all() and torch.isfinite(k).all()
