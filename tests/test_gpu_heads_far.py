"""GPU: operands whose rows lie further apart than 32-bit offsets reach give the
bits of the same operands side by side, and nothing between the rows changes."""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from train_helpers import normal

pytestmark = pytest.mark.gpu

ROWS, FAR = 300, 1 << 23          # 2.5e9 elements from the first row to the last
BF = torch.bfloat16


@pytest.fixture
def far():
    """A buffer of rows FAR apart, all 7, and a maker of (rows, heads, dim) views at columns that follow each other."""
    require_gpu()
    buffer = torch.full(((ROWS - 1) * FAR + (1 << 16),), 7.0, device="cuda", dtype=BF)
    at = [0]

    def view(like, fill=True):
        _, heads, dim = like.shape
        v = buffer.as_strided(like.shape, (FAR, dim, 1), at[0])
        at[0] += heads * dim + 64
        if fill:
            v.copy_(like)
        return v

    yield buffer, view
    del buffer
    torch.cuda.empty_cache()


def gaps_untouched(buffer, used):
    end = used + 4096
    rows = buffer[: (ROWS - 1) * FAR].view(ROWS - 1, FAR)
    return bool((rows[:, used:end] == 7.0).all()) and bool((rows[:, -4096:] == 7.0).all())


def test_attention(far):
    buffer, view = far
    q, k, v, dout = (normal(i, (ROWS, h, 80), BF) for i, h in enumerate((6, 2, 2, 6)))
    offsets = torch.tensor([0, 170, 171, ROWS], dtype=torch.int32, device="cuda")
    out, lse = nsmi.ns_attention(q, k, v, offsets)
    grads = nsmi.ns_attention_grad(dout, q, k, v, out, lse, offsets)
    fq, fk, fv, fg = (view(x) for x in (q, k, v, dout))
    fo = view(q, fill=False)
    got, got_lse = nsmi.ns_attention(fq, fk, fv, offsets, out=fo)
    assert torch.equal(got, out) and torch.equal(got_lse, lse)
    to = [view(x, fill=False) for x in (q, k, v)]
    for a, b in zip(nsmi.ns_attention_grad(fg, fq, fk, fv, fo, lse, offsets, dq=to[0], dk=to[1], dv=to[2]), grads):
        assert torch.equal(a, b)
    assert gaps_untouched(buffer, to[2].storage_offset() + 160)


def test_head_norm(far):
    buffer, view = far
    q, k, gq, gk = (normal(i, (ROWS, h, 128), BF) for i, h in enumerate((6, 2, 6, 2)))
    wq, wk = normal(8, (128,), BF), normal(9, (128,), BF)
    rest = (wq, wk, torch.arange(ROWS, device="cuda"), torch.rand(48, device="cuda"))
    want = nsmi.ns_qk_norm_rope(q, k, *rest)
    grads = nsmi.ns_qk_norm_rope_grad(gq, gk, q, k, *rest)
    fq, fk, fgq, fgk = (view(x) for x in (q, k, gq, gk))
    to = [view(x, fill=False) for x in (q, k, q, k)]
    for a, b in zip(nsmi.ns_qk_norm_rope(fq, fk, *rest, out_q=to[0], out_k=to[1]), want):
        assert torch.equal(a, b)
    for a, b in zip(nsmi.ns_qk_norm_rope_grad(fgq, fgk, fq, fk, *rest, dq=to[2], dk=to[3]), grads):
        assert torch.equal(a, b)
    assert gaps_untouched(buffer, to[3].storage_offset() + 256)


def test_token_logps(far):
    buffer, view = far
    logits = normal(3, (ROWS, 1, 1003), BF)
    tokens = torch.randint(0, 1003, (ROWS,), device="cuda")
    want = nsmi.ns_token_logps(logits[:, 0], tokens, top=3)
    d = normal(4, (ROWS,))
    grad = nsmi.ns_token_logps_grad(logits[:, 0], tokens, want[1], want[2], d, d)
    fz = view(logits)[:, 0]
    assert all(torch.equal(a, b) for a, b in zip(nsmi.ns_token_logps(fz, tokens, top=3), want))
    # (an output's rows may not lie between those of the logits)
    store = torch.full_like(buffer, 7.0)
    to = store.as_strided((ROWS, 1003), (FAR, 1), 5)
    assert torch.equal(nsmi.ns_token_logps_grad(fz, tokens, want[1], want[2], d, d, out=to), grad)
    assert gaps_untouched(store, 5 + 1003) and (store[:5] == 7.0).all()
    with pytest.raises(nsmi.NsError):
        nsmi.ns_token_logps_grad(fz, tokens, want[1], want[2], d, d, out=view(logits, fill=False)[:, 0])
    assert torch.equal(nsmi.ns_token_logps_grad(fz, tokens, want[1], want[2], d, d, out=fz), grad)
    assert gaps_untouched(buffer, 2 * (1003 + 64))
