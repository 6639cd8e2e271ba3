"""The most rows, sequences and heads of an attention call: the calls and their
workspace sizes draw the same line, and the GPU runs what lies on it."""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from test_heads_abi import BAD, MB, P, UNSUPPORTED, attn

HEADS, KEY_HEADS, DIM, MOST = 32, 2, 16, 130055   # MOST sequences of a token each

# tokens, sequences: (tokens / 128 + sequences + 1) * 32 is 2^22 or the multiple before it, then beyond
BORDER = [(MOST, MOST, True), (MOST, MOST + 1, False), (1, 131071, True), (1, 131072, False),
          (1 << 23, 65535, True), (1 << 23, 65536, False), (127, 131071, True), (128, 131071, False)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
@pytest.mark.parametrize("tokens, sequences, inside", BORDER)
def test_both_sides_of_the_border(tokens, sequences, inside):
    assert ((tokens // 128 + sequences + 1) * HEADS <= nsmi.NS_MAX_HEAD_TILES) == inside
    far = [P[0] + i * (1 << 40) for i in range(11)]   # further apart than the tensors are long
    wide, narrow = (HEADS * DIM, DIM), (KEY_HEADS * DIM, DIM)
    places = dict(q=(far[0], *wide), k=(far[1], *narrow), v=(far[2], *narrow), offsets=far[3], lse=far[4],
                  out=(far[5], *wide), dout=(far[6], *wide), dq=(far[7], *wide), dk=(far[8], *narrow),
                  dv=(far[9], *narrow), ws=far[10], n=1 << 39)
    for call, size in (("forward", nsmi.ns_attention_workspace_size), ("grad", nsmi.ns_attention_grad_workspace_size)):
        found = attn(call, tokens=tokens, sequences=sequences, q_heads=HEADS, k_heads=KEY_HEADS, dim=DIM, **places)
        assert found == (UNSUPPORTED if inside else BAD)
        if inside:
            assert size(tokens, sequences, HEADS, KEY_HEADS, DIM) >= 0
        else:
            with pytest.raises(nsmi.NsError):
                size(tokens, sequences, HEADS, KEY_HEADS, DIM)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
def test_without_tokens_there_is_no_border():
    for call in ("forward", "grad"):
        assert attn(call, tokens=0, sequences=nsmi.NS_MAX_ROWS, q_heads=1024, k_heads=1024) == nsmi.NS_OK
    assert nsmi.ns_attention_workspace_size(0, nsmi.NS_MAX_ROWS, 1024, 1024, 128) >= 0


@pytest.mark.gpu
def test_as_many_sequences_as_there_may_be():
    """A token each: out is v, dq and dk are 0 and dv is the sum of a group's dout."""
    require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(3)

    def some(heads):
        return torch.randint(-8, 9, (MOST, heads, DIM), generator=gen, device="cuda").to(torch.bfloat16)

    q, k, v, dout = some(HEADS), some(KEY_HEADS), some(KEY_HEADS), some(HEADS)
    ends = torch.arange(MOST + 1, dtype=torch.int32, device="cuda")
    out, lse = nsmi.ns_attention(q, k, v, ends)
    assert torch.equal(out, v.repeat_interleave(HEADS // KEY_HEADS, 1))
    dq, dk, dv = nsmi.ns_attention_grad(dout, q, k, v, out, lse, ends)
    # P = exp(S - lse) is 1 but for fp32's roundings; dout . out and delta are the same whole numbers
    assert not dq.any() and not dk.any()
    want = dout.float().unflatten(1, (KEY_HEADS, -1)).sum(2)
    assert ((dv.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -8 * 16 * 8).all()
