"""GPU: lse of long rows of attention whose scores differ widely: the small weights are many,
and each below half a step of the row's whole sum.

Tolerance. Scores of deviation 4 and 8, lse between 16 and 64: lse itself is rounded by up to half a
step, 2^-20 below 32, and S by fp32 sums of 128 products, to both sides and apart in every row. The mean
over 512 rows may be off by half of lse's step, no more; what a sum in fp32 loses always lies on one side."""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens, heads, dim, dtype, size", [
    (16384, 32, 128, torch.bfloat16, 4.0),   # 64 queries a wave
    (16384, 4, 128, torch.float16, 4.0),     # parts
    (8192, 4, 64, torch.bfloat16, 4.0),
    (8192, 12, 96, torch.bfloat16, 4.0), (12000, 2, 128, torch.bfloat16, 4.0)], ids=str)
def test_small_weights_are_not_lost_beside_long_sums(tokens, heads, dim, dtype, size):
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = (torch.randn((tokens, heads, dim), generator=gen, device="cuda") * size).to(dtype)
    k, v = (torch.randn((tokens, 1, dim), generator=gen, device="cuda").to(dtype) for _ in range(2))
    _, lse = nsmi.ns_attention(q, k, v, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"))
    rows = torch.arange(tokens - 512, tokens, device="cuda")
    scores = q[rows, 0].double() @ k[:, 0].double().t().contiguous() * dim ** -0.5
    scores.masked_fill_(torch.arange(tokens, device="cuda") > rows[:, None], float("-inf"))
    want = torch.logsumexp(scores, -1)
    assert 8 < want.mean() < 32
    off = (lse[0, rows].double() - want).mean().item()
    assert abs(off) < 2.0 ** -20, off * 2.0 ** 24
