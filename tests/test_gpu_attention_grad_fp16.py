"""GPU: the gradient of fp16 attention where sequences and heads differ widely in size:
each is as exact as it is alone, whatever lies beside it.

Tolerances. Those of the gradient's other tests: weights off by e_p and half a step of
fp16 each, dS the same, dout . v and delta sums of dim terms in fp32. Beyond them a dS
among fp16's subnormals is off by 2^-25 of a range whose 2^13 is at most what a dS of
its own sequence and group of heads can reach, 2 |dout| |v|; and a weight by 2^-25 of 2^14."""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import heads_oracle as H
from test_gpu_attention import make, weight_error
from train_helpers import U32, assert_within, f64, half_step, normal

pytestmark = pytest.mark.gpu

HF = torch.float16
LENGTHS, HEADS, KEY_HEADS = [120, 0, 333, 1, 200], 4, 2
SCALE = 2.0 ** 15   # of scores whose queries and keys are of size 2^-9


def gradients(c, dout):
    out, lse = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"], scale=SCALE)
    return out, lse, nsmi.ns_attention_grad(dout, c["q"], c["k"], c["v"], out, lse, c["offsets"], scale=SCALE)


def check_part(c, dout, out, lse, got, a, b, head):
    """Rows a .. b (a whole sequence) and the group of key head `head` against the oracle."""
    group = c["q"].shape[1] // c["k"].shape[1]
    mine, dim = slice(head * group, (head + 1) * group), c["q"].shape[2]
    n = b - a
    part = dict(q=c["q"][a:b, mine], k=c["k"][a:b, head:head + 1], v=c["v"][a:b, head:head + 1])
    args = [f64(dout[a:b, mine]), *(f64(part[x]) for x in "qkv"), f64(out[a:b, mine]), f64(lse[mine, a:b])]
    rel = 2 * weight_error(part, [0, n], SCALE, args[5]) + 2.0 ** -11 + (group * n / 16 + 8) * U32
    want, slack = H.attention_grad(*args, [0, n], SCALE, rel=rel, dp_err=(2 * dim + 8) * U32)
    norm = lambda x: np.sqrt((x ** 2).sum(-1).max())   # noqa: E731
    reach = 2 * SCALE * norm(args[0]) * norm(args[3])
    for name, g, w, sl, other, of in (("dq", got[0][a:b, mine], want[0], slack[0], args[2], reach),
                                      ("dk", got[1][a:b, head:head + 1], want[1], slack[1], args[1], reach),
                                      ("dv", got[2][a:b, head:head + 1], want[2], slack[2], args[0], 1.0)):
        tiny = n * group * np.abs(other).max() * 2.0 ** -38 * of
        g, sl = f64(g), half_step(w, HF) + sl + tiny
        # (from 65520 on, half a step past the type's largest, numbers round to infinity)
        g = np.where(np.isinf(g) & (g * w > 0) & (np.abs(w) + sl >= 65520), w, g)
        assert_within(g, w, sl, f"{name} of rows {a} to {b}, key head {head}")


def sequences(lengths):
    ends = np.concatenate([[0], np.cumsum(lengths)])
    return [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:]) if b > a]


def small(seed, lengths, heads, key_heads, dim):
    """A batch whose dS, 10^-7 or so, would hardly be told from 0 in fp16 as it stands. Its gradients
    are 10^-4 or so: of scores of size 1 from small queries and keys and a large scale."""
    c = make(seed, lengths, heads, key_heads, dim, HF)
    c["k"] *= 2.0 ** -9
    c["q"] *= 2.0 ** -9
    return c, normal(seed + 9, c["q"].shape, HF, 2e-6)


@pytest.mark.parametrize("dim", [64, 80])
@pytest.mark.parametrize("what", ["inf in dout", "inf in v", "nan in dout", "nan in v"])
def test_not_finite_in_another_sequence(what, dim):
    require_gpu()
    c, dout = small(1, LENGTHS, HEADS, KEY_HEADS, dim)
    value, name = what.split(" in ")
    a, b = 120, 453
    (dout if name == "dout" else c["v"])[a + 70, 1, 3] = float(value)
    out, lse, got = gradients(c, dout)
    assert not torch.isfinite(got[0][a:b]).all() and not torch.isfinite(got[1][a:b]).all()
    for first, last in sequences(LENGTHS):
        if first != a:
            for head in range(KEY_HEADS):
                check_part(c, dout, out, lse, got, first, last, head)
    # the other group of heads of the same sequence has none of it
    check_part(c, dout, out, lse, got, a, b, 1 if name == "dout" else 0)


@pytest.mark.parametrize("lengths", [LENGTHS, [1100, 37, 200]], ids=str)
@pytest.mark.parametrize("name", ["dout", "v"])
def test_large_rows_elsewhere(name, lengths):
    """A row that is much larger: in another sequence, and in another group of heads. (1100
    rows: few workgroups, cut into parts.)"""
    require_gpu()
    c, dout = small(2, lengths, HEADS, KEY_HEADS, 64)
    t = dout if name == "dout" else c["v"]
    parts = sequences(lengths)
    a, b = parts[-1]
    t[a + 50, 0] *= 1e8 if name == "dout" else 1e4      # (v itself is of size 1)
    out, lse, got = gradients(c, dout)
    for first, last in parts[:-1]:
        for head in range(KEY_HEADS):
            check_part(c, dout, out, lse, got, first, last, head)
    check_part(c, dout, out, lse, got, a, b, 1)


def test_alone_and_beside_others():
    """A sequence alone and beside one of a hundred million times its size: the same bits of dq. (dk
    and dv of the whole batch, whose 654 rows of two heads a group are 1308, are cut into
    two parts, the sequences' alone into one: their sums have another order.)"""
    require_gpu()
    c, dout = small(3, LENGTHS, HEADS, KEY_HEADS, 128)
    dout[454:] *= 1e8
    out, lse, got = gradients(c, dout)
    for a, b in sequences(LENGTHS):
        one = {x: c[x][a:b].contiguous() for x in "qkv"}
        ends = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        rest = (dout[a:b].contiguous(), out[a:b].contiguous(), lse[:, a:b].contiguous())
        alone = nsmi.ns_attention_grad(rest[0], one["q"], one["k"], one["v"], *rest[1:], ends, scale=SCALE)
        assert torch.equal(alone[0], got[0][a:b])
        for head in range(KEY_HEADS):
            check_part(one, *rest, alone, 0, b - a, head)
            check_part(c, dout, out, lse, got, a, b, head)


def test_rows_of_one_sequence():
    """dq of small rows behind a large one of the same sequence and head: each row has a range of its own."""
    require_gpu()
    c, dout = small(4, [400], 2, 1, 64)
    dout[0, 0] *= 1e8
    out, lse, got = gradients(c, dout)
    args = [f64(x) for x in (dout, c["q"], c["k"], c["v"], out, lse)]
    rel = 2 * weight_error(c, [0, 400], SCALE, args[5]) + 2.0 ** -11 + (2 * 400 / 16 + 8) * U32
    want, slack = H.attention_grad(*args, [0, 400], SCALE, rel=rel, dp_err=(2 * 64 + 8) * U32)
    norm = lambda x: np.sqrt((x ** 2).sum(-1))   # noqa: E731
    reach = 2 * SCALE * norm(args[0])[..., None] * norm(args[3]).max()   # each row's
    tiny = 400 * np.abs(args[2]).max() * 2.0 ** -38 * reach
    assert_within(got[0], want[0], half_step(want[0], HF) + slack[0] + tiny, "dq")
