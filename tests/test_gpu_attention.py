"""GPU: causal attention over packed sequences and its gradient against the fp64
oracle.

Tolerances. S is a sum of dim products in fp32: off by at most dim half steps of
the products' magnitudes (sq_err), and its exponent by 4 half steps of the largest
|S| or |lse|; a weight is then off by e_p = sq_err + those, relative, and by half a
step of its type where it goes into a product. An output is that of its weights,
plus the fp32 sum over the keys (one half step a matrix instruction of 16 keys, at
most n / 16 + 8 of them), plus its own rounding. The gradient is measured from the
given out and lse, dout . v and delta each a sum of dim terms in fp32."""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import heads_oracle as H
from train_helpers import U32, assert_within, f64, half_step, normal

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def ends_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def make(seed, lengths, q_heads, k_heads, dim, dtype, rest=0, peak=1.0):
    t = sum(lengths) + rest
    c = dict(q=normal(seed, (t, q_heads, dim), dtype, peak), k=normal(seed + 1, (t, k_heads, dim), dtype),
             v=normal(seed + 2, (t, k_heads, dim), dtype), offsets=ends_of(lengths))
    if rest:
        for x in ("q", "k", "v"):   # what lies behind the last sequence is not read
            c[x][t - rest:] = float("nan")
    return c


def weight_error(c, ends, scale, lse):
    """Most that a weight may be off, relative, but for its rounding."""
    dim = c["q"].shape[2]
    n = ends[-1]
    norm = lambda x: np.sqrt((f64(x)[:n] ** 2).sum(-1).max(initial=0.0))   # noqa: E731
    most = scale * norm(c["q"]) * norm(c["k"])
    return (dim + 8) * U32 * most + 4 * U32 * np.abs(lse).max(initial=0.0) + 16 * U32


def check(c, scale=None, times=1, **outs):
    """(times: the heads that many times one behind the other, which must all come out alike.)"""
    dtype, dim = c["q"].dtype, c["q"].shape[2]
    out, lse = nsmi.ns_attention(*(c[x].repeat(1, times, 1) if times > 1 else c[x] for x in "qkv"), c["offsets"],
                                 scale=scale, **outs)
    if times > 1:
        outs_of, lses = out.unflatten(1, (times, -1)), lse.unflatten(0, (times, -1))
        assert (outs_of == outs_of[:, :1]).all() and (lses == lses[:1]).all()
        out, lse = outs_of[:, 0], lses[0]
    ends = c["offsets"].tolist()
    s = dim ** -0.5 if scale is None else scale
    n = ends[-1]
    want, want_lse, spread = H.attention(*(np.nan_to_num(f64(c[x])) for x in "qkv"), ends, s)
    e_p = weight_error(c, ends, s, want_lse)
    longest = max(b - a for a, b in zip(ends[:-1], ends[1:])) if len(ends) > 1 else 0
    step = torch.finfo(dtype).eps / 2
    slack = half_step(want, dtype) + (2 * e_p + step + (longest / 16 + 8) * U32) * spread
    if dtype == HF:   # weights among the subnormals: 2^-25 of a scale that is at most 2^-7 of the largest
        slack = slack + longest * 2.0 ** -32 * np.abs(np.nan_to_num(f64(c["v"]))).max(initial=0.0)
    assert_within(out[:n], want[:n], slack[:n], "out")
    assert_within(lse[:, :n], want_lse[:, :n], e_p + (longest / 32 + 16) * U32 + half_step(want_lse, lse.dtype)[:, :n], "lse")
    return out, lse


CASES = [
    # lengths, q_heads, k_heads, dim
    ([1], 1, 1, 64), ([2, 1, 0, 3], 4, 2, 128), ([64], 2, 1, 128), ([65, 63], 3, 3, 64), ([127, 1, 129], 4, 1, 128),
    ([200], 8, 8, 80), ([31, 33, 0, 0, 97, 5], 6, 2, 8), ([513], 2, 2, 72), ([300, 40], 16, 8, 128),
    ([0, 0, 7], 2, 1, 16), ([130, 257, 61], 12, 4, 112), ([1000], 1, 1, 56), ([1] * 150, 2, 1, 64),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c)[:40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward(case, dtype):
    require_gpu()
    lengths, *shape = case
    check(make(len(lengths) + sum(lengths), lengths, *shape, dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_peaked_and_flat(dtype):
    require_gpu()
    check(make(1, [400, 77], 4, 2, 128, dtype, peak=30.0))
    check(make(2, [400, 77], 4, 2, 64, dtype), scale=2.0)
    check(make(3, [333], 4, 2, 64, dtype), scale=1e-4)
    c = make(4, [300], 2, 1, 64, dtype)
    c["q"] *= 0           # every key the same
    check(c)
    c = make(5, [300], 2, 1, 64, dtype)
    # scores that rise along the sequence: the reference moves with every tile
    c["k"][:, 0] = torch.linspace(0, 4, 300, device="cuda").to(dtype)[:, None]
    c["q"][:] = 2.0
    check(c)
    c["k"] = c["k"].flip(0).contiguous()
    check(c)


# Rows of all heads from 294912 on, 512 or more a sequence: waves take 64 queries for heads above 64.
@pytest.mark.parametrize("lengths, rest, dim", [([577], 0, 128), ([513, 1100], 0, 72), ([1400, 0, 301], 61, 104),
                                                ([2049], 0, 64), ([1, 1, 2300], 1, 128)], ids=str)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_many_queries(lengths, rest, dim, dtype):
    require_gpu()
    c = make(9, lengths, 4, 2, dim, dtype, rest=rest)
    times = -(-294912 // (4 * c["q"].shape[0]))
    out, lse = check(c, times=times)
    n = sum(lengths)
    assert not out[n:].any() and not lse[:, n:].any()
    c = make(10, lengths, 4, 2, dim, dtype, peak=30.0)
    c["k"][:, 1] = torch.linspace(0, 4, n, device="cuda").to(dtype)[:, None]
    check(c, times=times)


# From 512 workgroups of short sequences on, or 1024: tiles of 32 keys for heads above 64.
@pytest.mark.parametrize("lengths, rest, dim, heads", [([130, 1, 0, 64, 200, 33], 0, 128, 52), ([700], 0, 72, 148),
                                                       ([31, 32, 33, 63, 65, 257], 70, 96, 64),
                                                       ([1] * 70 + [129, 40], 1, 128, 8), ([640, 389], 5, 120, 96)], ids=str)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_many_workgroups(lengths, rest, dim, heads, dtype):
    require_gpu()
    c = make(11, lengths, 4, 2, dim, dtype, rest=rest)
    out, lse = check(c, times=heads // 4)
    n = sum(lengths)
    assert not out[n:].any() and not lse[:, n:].any()
    c = make(12, lengths, 4, 2, dim, dtype, peak=30.0)
    check(c, times=heads // 4)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_behind_the_last_sequence(dtype):
    require_gpu()
    for rest in (1, 130, 700):
        c = make(6, [100, 30], 4, 2, 72, dtype, rest=rest)
        out, lse = check(c)
        assert not out[130:].any() and not lse[:, 130:].any()
        given = torch.full_like(c["q"], 7.0)
        again, _ = check(c, out=given)
        assert again.data_ptr() == given.data_ptr()
        assert (given[130:] == 7.0).all() and torch.equal(given[:130], out[:130])


def test_no_sequences_and_no_tokens():
    require_gpu()
    c = make(7, [], 2, 1, 64, BF, rest=40)
    out, lse = check(c)
    assert not out.any() and not lse.any()
    c = make(7, [0, 0], 2, 1, 64, BF)
    out, lse = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"])
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    grads = nsmi.ns_attention_grad(out, c["q"], c["k"], c["v"], out, lse, c["offsets"])
    assert [g.shape[0] for g in grads] == [0, 0, 0]


def fused(c):
    """q, k and v as parts of one projection's output."""
    t, hq, d = c["q"].shape
    hk = c["k"].shape[1]
    both = torch.cat([c["q"], c["k"], c["v"]], 1)
    return dict(c, q=both[:, :hq], k=both[:, hq:hq + hk], v=both[:, hq + hk:])


@pytest.mark.parametrize("dim", [64, 120, 128])
def test_other_layouts(dim):
    require_gpu()
    c = make(8, [70, 150, 3], 4, 2, dim, BF)
    want = check(c)
    got = check(fused(c))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    by_head = {x: c[x].transpose(0, 1).contiguous().transpose(0, 1) for x in "qkv"}
    got = check(dict(by_head, offsets=c["offsets"]), out=torch.empty_like(by_head["q"]))
    assert got[0].stride(0) == dim
    assert torch.equal(got[0], want[0])
    one = dict(c, k=c["k"][:, :1].expand(-1, 2, -1), v=c["v"][:, :1].expand(-1, 2, -1))
    got = nsmi.ns_attention(one["q"], one["k"], one["v"], c["offsets"])
    want = nsmi.ns_attention(c["q"], c["k"][:, :1].contiguous(), c["v"][:, :1].contiguous(), c["offsets"])
    assert torch.equal(got[0], want[0])


def test_sequences_do_not_see_each_other():
    """A NaN or infinity stays in its sequence; each sequence alone gives the same bits."""
    require_gpu()
    lengths = [50, 129, 64, 200]
    c = make(9, lengths, 4, 2, 128, BF)
    out, lse = check(c)
    ends = c["offsets"].tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        alone = nsmi.ns_attention(*(c[x][a:b].contiguous() for x in "qkv"), ends_of([b - a]))
        assert torch.equal(alone[0], out[a:b]) and torch.equal(alone[1], lse[:, a:b])
    bad = dict(c, **{x: c[x].clone() for x in "qkv"})
    bad["k"][60], bad["v"][100], bad["v"][178], bad["q"][70] = float("nan"), float("inf"), float("nan"), float("nan")
    got, got_lse = nsmi.ns_attention(bad["q"], bad["k"], bad["v"], c["offsets"])
    for a, b in ((0, 50), (179, 443)):
        assert torch.equal(got[a:b], out[a:b]) and torch.equal(got_lse[:, a:b], lse[:, a:b])


def check_grad(c, scale=None, seed=50, size=0.1, **given):
    dtype, dim = c["q"].dtype, c["q"].shape[2]
    s = dim ** -0.5 if scale is None else scale
    dout = normal(seed, c["q"].shape, dtype, size)
    ends = c["offsets"].tolist()
    n = ends[-1]
    dout[n:] = float("nan")
    out, lse = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"], scale=scale)
    got = nsmi.ns_attention_grad(dout, c["q"], c["k"], c["v"], out, lse, c["offsets"], scale=scale, **given)
    clean = lambda t: np.nan_to_num(f64(t))   # noqa: E731
    e_p = weight_error(c, ends, s, f64(lse)[:, :n])
    step = torch.finfo(dtype).eps / 2
    longest = max((b - a for a, b in zip(ends[:-1], ends[1:])), default=0)
    group = c["q"].shape[1] // c["k"].shape[1]
    sums = (group * longest / 16 + 8) * U32
    args = (clean(dout), clean(c["q"]), clean(c["k"]), clean(c["v"]), clean(out), clean(lse))
    want, slack = H.attention_grad(*args, ends, s, rel=2 * e_p + step + sums, dp_err=(2 * dim + 8) * U32)
    for name, g, w, sl in zip(("dq", "dk", "dv"), got, want, slack):
        assert g.dtype == dtype
        tiny = 0.0
        if w.size:
            # fp16: dS among the subnormals of the scaled range, 2^-25 where the largest possible is 2^13 or more;
            # a weight or a dS below fp32's normal range, 2^-126, is 0, each of them at most once
            norm = lambda x: np.sqrt((x[:n] ** 2).sum(-1).max(initial=0.0))   # noqa: E731
            other = {"dq": args[2], "dk": args[1], "dv": args[0]}[name]
            least = 2.0 ** -38 if dtype == HF else 2.0 ** -125
            tiny = longest * group * np.abs(other).max() * least * max(2 * s * norm(args[0]) * norm(args[3]), 1.0)
        assert_within(g[:n], w[:n], half_step(w, dtype)[:n] + sl[:n] + tiny, name)
    return dout, out, lse, got


@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c)[:40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradient(case, dtype):
    require_gpu()
    lengths, *shape = case
    check_grad(make(len(lengths) + sum(lengths) + 3, lengths, *shape, dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradient_sizes(dtype):
    """Large and small gradients (fp16: dS below its range as it stands), peaked weights."""
    require_gpu()
    c = make(11, [260, 90], 4, 2, 64, dtype)
    check_grad(c, size=1e-4)
    check_grad(c, size=50.0)
    check_grad(make(12, [260, 90], 4, 2, 128, dtype, peak=20.0))
    check_grad(make(13, [260, 90], 4, 2, 128, dtype), scale=1.5)
    dout, out, lse, _ = check_grad(c)
    zero = nsmi.ns_attention_grad(dout * 0, c["q"], c["k"], c["v"], out, lse, c["offsets"])
    assert not any(g.any() for g in zero)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradient_behind_the_last_sequence(dtype):
    require_gpu()
    for rest in (1, 200):
        c = make(14, [100, 30], 4, 2, 72, dtype, rest=rest)
        dout, out, lse, got = check_grad(c)
        assert not any(g[130:].any() for g in got)
        store = torch.full((130 + rest, 8, 72), 7.0, dtype=dtype, device="cuda")
        parts = dict(dq=store[:, :4], dk=store[:, 4:6], dv=store[:, 6:])
        given = nsmi.ns_attention_grad(dout, c["q"], c["k"], c["v"], out, lse, c["offsets"], **parts)
        assert all(torch.equal(a[:130], b[:130]) for a, b in zip(given, got))
        assert (store[130:] == 7.0).all()


def test_gradient_of_other_layouts_and_alone():
    require_gpu()
    lengths = [70, 150, 3]
    c = make(15, lengths, 4, 2, 128, BF)
    dout, out, lse, want = check_grad(c)
    f = fused(c)
    g = dout.transpose(0, 1).contiguous().transpose(0, 1)
    got = nsmi.ns_attention_grad(g, f["q"], f["k"], f["v"], out, lse, c["offsets"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ends = c["offsets"].tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        alone = nsmi.ns_attention_grad(*(x[a:b].contiguous() for x in (dout, c["q"], c["k"], c["v"], out)),
                                       lse[:, a:b].contiguous(), ends_of([b - a]))
        assert all(torch.equal(x, y[a:b]) for x, y in zip(alone, want))


@pytest.mark.parametrize("case", [([1100, 37, 200], 4, 2, 128), ([1300], 2, 1, 64), ([3, 0, 1500, 90], 6, 2, 80),
                                  ([700] * 3, 3, 3, 120)], ids=lambda c: str(c)[:40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_long_sequences(case, dtype):
    """Where few workgroups are cut into parts, whose sums are brought together."""
    require_gpu()
    lengths, *shape = case
    c = make(sum(lengths), lengths, *shape, dtype, rest=5)
    assert nsmi.ns_attention_workspace_size(len(c["q"]), len(lengths), *shape) > 0
    check(c)
    check_grad(c)
    peaked = make(1, lengths, *shape, dtype, peak=25.0)
    check(peaked)
    check_grad(peaked)
    ws = torch.full((nsmi.ns_attention_workspace_size(len(c["q"]), len(lengths), *shape),), 255, dtype=torch.uint8,
                    device="cuda")
    out, lse = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"], workspace=ws)
    again, lse2 = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"])
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_offsets_that_do_not_rise():
    """No row outside the tensors is touched, whatever the offsets hold."""
    require_gpu()
    store = torch.full((3, 300, 4, 64), 7.0, dtype=BF, device="cuda")
    c = make(16, [300], 4, 4, 64, BF)
    for ends in ([0, 400], [-5, 100, 300], [0, 200, 100, 1 << 30], [5, 3], [-(1 << 31), (1 << 31) - 1], [300, 0]):
        offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
        out = store[1].fill_(7.0)
        nsmi.ns_attention(c["q"], c["k"], c["v"], offsets, out=out)
        lse = torch.zeros((4, 300), device="cuda")
        dq, dk, dv = (torch.empty_like(c["q"]) for _ in range(3))
        nsmi.ns_attention_grad(c["q"], c["q"], c["k"], c["v"], c["q"], lse, offsets, dq=dq, dk=dk, dv=dv)
        torch.cuda.synchronize()
        assert (store[0] == 7.0).all() and (store[2] == 7.0).all()


def test_long_sequence_samples():
    """A long sequence: rows at its ends and middle, against 64 bits."""
    require_gpu()
    n, d = 9001, 128
    c = make(17, [n], 2, 1, d, BF)
    out, lse = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"])
    q, k, v = (f64(c[x]) for x in "qkv")
    e_p = weight_error(c, [0, n], d ** -0.5, np.array([12.0]))
    for i in (0, 1, 63, 64, 127, 128, 4500, 8959, 8960, 9000):
        for h in range(2):
            s = k[:i + 1, 0] @ q[i, h] * d ** -0.5
            p = np.exp(s - s.max())
            want = p @ v[:i + 1, 0] / p.sum()
            spread = p @ np.abs(v[:i + 1, 0]) / p.sum()
            slack = half_step(want, BF) + (2 * e_p + 2.0 ** -8 + (n / 16 + 8) * U32) * spread
            assert_within(out[i, h], want, slack, f"row {i}")
            assert abs(lse[h, i].item() - s.max() - np.log(p.sum())) < e_p + (n / 32 + 32) * U32 + 12 * U32
