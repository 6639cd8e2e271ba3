"""GPU: what a NaN or infinity in one sequence does to the gradients of the others: nothing,
to the bit."""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from test_gpu_attention import make
from train_helpers import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths, heads, dim", [([50, 129, 64, 200], (4, 2), 128), ([1300, 40, 700], (2, 1), 80),
                                                 ([3, 31, 1, 33, 0, 7], (8, 8), 64)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_other_sequences_keep_their_bits(lengths, heads, dim, value, dtype):
    require_gpu()
    c = make(sum(lengths), lengths, *heads, dim, dtype)
    dout = normal(7, c["q"].shape, dtype, 0.1)

    def gradients():
        out, lse = nsmi.ns_attention(c["q"], c["k"], c["v"], c["offsets"])
        return out, nsmi.ns_attention_grad(dout, c["q"], c["k"], c["v"], out, lse, c["offsets"])

    out, want = gradients()
    a, b = lengths[0], lengths[0] + lengths[1]   # the second sequence's first, middle and last rows
    for t in (c["q"], c["k"], c["v"], dout):
        kept = t[a:b].clone()
        for row in {a, (a + b) // 2, b - 1}:
            t[row, 0, 2] = value
            got_out, got = gradients()
            for x, y in zip((out, *want), (got_out, *got)):
                assert torch.equal(x[:a], y[:a]) and torch.equal(x[b:], y[b:])
            t[a:b] = kept
    again = gradients()
    assert torch.equal(again[0], out) and all(torch.equal(x, y) for x, y in zip(again[1], want))
