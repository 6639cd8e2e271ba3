"""Refusals of the operators on heads and of the token log probabilities, at the C
ABI and in the binding, without a GPU: bad arguments are answered before any device
work (the addresses here belong to nothing and are never touched), and valid ones
reach the device check."""

import ctypes
import os

import pytest

import newton_schulz_matrix_amd as nsmi
from newton_schulz_matrix_amd import heads
from newton_schulz_matrix_amd import operators as ops

pytestmark = pytest.mark.skipif(not os.path.exists(nsmi.LIB_PATH), reason="libnsmi.so not built")

BAD, UNSUPPORTED, WS = nsmi.NS_ERR_INVALID_ARG, nsmi.NS_ERR_UNSUPPORTED, nsmi.NS_ERR_WORKSPACE
F32, BF16, F16, E4M3 = nsmi.NS_DT_F32, nsmi.NS_DT_BF16, nsmi.NS_DT_F16, nsmi.NS_DT_E4M3
MB = 1 << 20
P = [(64 + 64 * i) * MB for i in range(20)]   # addresses 64 MB apart
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")


def logps(call="forward", ws=P[8], n=64 * MB, lse=P[3], entropy=P[4], logps=P[5], top_logps=P[6], top_ids=P[7],
          dlogps=P[5], dentropy=P[6], out=P[9], ld_out=100, **kw):
    a = dict(logits=P[0], tokens=P[1], rows=8, vocab=100, ld=100, top=3, dtype=BF16, token_type=1, length=0,
             ld_sequence=0)
    a.update(kw)
    args = ctypes.byref(ops._TokenLogpsArgs(*a.values()))
    if call == "forward":
        return nsmi.library().ns_token_logps(args, logps, lse, entropy, top_logps, top_ids, ws, n, None)
    return nsmi.library().ns_token_logps_grad(args, lse, entropy, dlogps, dentropy, out, ld_out, None)


def test_token_logps_refusals():
    lib = nsmi.library()
    assert lib.ns_token_logps(None, *P[2:7], P[8], MB, None) == BAD
    assert lib.ns_token_logps_grad(None, *P[2:6], P[7], 100, None) == BAD
    for call in ("forward", "grad"):
        assert logps(call) == UNSUPPORTED
        assert logps(call, rows=0, logits=None, tokens=None) == nsmi.NS_OK
        assert logps(call, token_type=0, tokens=P[1] + 4) == UNSUPPORTED
        assert logps(call, logits=P[0] + 2, ld=101) == UNSUPPORTED     # element alignment is enough
        assert logps(call, length=4, ld_sequence=500) == UNSUPPORTED and logps(call, length=4) == UNSUPPORTED
        assert logps(call, length=8, ld_sequence=1) == UNSUPPORTED     # one sequence: its distance does not count
        for kw in (dict(length=3), dict(length=-4), dict(length=16), dict(length=4, ld_sequence=399),
                   dict(length=4, ld_sequence=-400), dict(length=4, ld_sequence=1 << 60), dict(length=1 << 40)):
            assert logps(call, **kw) == BAD, (call, kw)
        for kw in (dict(logits=None), dict(tokens=None), dict(lse=None), dict(rows=-1), dict(vocab=0),
                   dict(rows=nsmi.NS_MAX_ROWS + 1), dict(vocab=nsmi.NS_MAX_ROWS + 1, ld=1 << 30), dict(ld=99),
                   dict(ld=1 << 40), dict(dtype=E4M3), dict(dtype=-1), dict(token_type=2), dict(top=-1),
                   dict(top=65), dict(top=3, vocab=2), dict(logits=P[0] + 1), dict(tokens=P[1] + 4),
                   dict(lse=P[3] + 2), dict(entropy=P[4] + 1)):
            assert logps(call, **kw) == BAD, (call, kw)
    assert logps(top=0, top_logps=None, top_ids=None) == UNSUPPORTED
    for kw in (dict(logps=None), dict(entropy=None), dict(top_logps=None), dict(top_ids=None), dict(top=0),
               dict(top_ids=P[7] + 4), dict(top_logps=P[6] + 2), dict(logps=P[3]), dict(lse=P[0]),
               dict(top_ids=P[1]), dict(top_logps=P[7] + 8)):
        assert logps(**kw) == BAD, kw
    cut = dict(rows=2, vocab=40000, ld=40000)      # few long rows are cut into pieces; others need no workspace
    for kw in (dict(ws=None), dict(n=8), dict(ws=P[8] + 64)):
        assert logps(**cut, **kw) == WS and logps(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=P[0]), dict(ws=P[6]), dict(ws=P[7])):
        assert logps(**cut, **kw) == BAD, kw
    assert logps("grad", out=P[0]) == UNSUPPORTED                      # in place
    assert logps("grad", out=P[0], length=2, ld_sequence=8 * MB) == UNSUPPORTED
    assert logps("grad", out=P[0] + 32 * MB, length=2, ld_sequence=8 * MB) == BAD   # in the last sequence
    assert logps("grad", out=P[0] + 56 * MB, length=2, ld_sequence=8 * MB) == UNSUPPORTED
    assert logps("grad", dentropy=None, entropy=None) == UNSUPPORTED
    assert logps("grad", dlogps=None) == UNSUPPORTED
    for kw in (dict(out=None), dict(entropy=None), dict(ld_out=99), dict(out=P[0], ld_out=104), dict(out=P[0] + 2),
               dict(out=P[1]), dict(out=P[3]), dict(out=P[4]), dict(out=P[5]), dict(out=P[6]), dict(out=P[9] + 1),
               dict(dlogps=P[5] + 2), dict(dentropy=P[6] + 2)):
        assert logps("grad", **kw) == BAD, kw


def part(data, token, head):
    return heads._Heads(data, token, head)


def qk(call="forward", q_out=None, k_out=None, dq_out=None, dk_out=None, dqw=P[14], dkw=P[15], dw=F32, ws=P[16],
       n=64 * MB, **kw):
    a = dict(q=(P[0], 512, 128), k=(P[1], 256, 128), q_weight=P[2], k_weight=P[3], positions=P[4], inv_freq=P[5],
             tokens=6, q_heads=4, k_heads=2, dim=128, rotary=64, ld_positions=0, axes=1, sections=(0, 0, 0, 0),
             interleaved=0, dtype=BF16, weight_dtype=F32, position_type=1, eps=1e-6)
    a.update(kw)
    args = ctypes.byref(heads._QkNormRopeArgs(**a))
    q_out, k_out = part(*(q_out or (P[6], 512, 128))), part(*(k_out or (P[7], 256, 128)))
    if call == "forward":
        return nsmi.library().ns_qk_norm_rope(args, q_out, k_out, None)
    dq_out, dk_out = part(*(dq_out or (P[8], 512, 128))), part(*(dk_out or (P[9], 256, 128)))
    return nsmi.library().ns_qk_norm_rope_grad(args, dq_out, dk_out, q_out, k_out, dqw, dkw, dw, ws, n, None)


def test_qk_norm_rope_refusals():
    lib = nsmi.library()
    one = part(P[0], 512, 128)
    assert lib.ns_qk_norm_rope(None, one, one, None) == BAD
    assert lib.ns_qk_norm_rope_grad(None, one, one, one, one, P[1], P[2], 0, P[3], MB, None) == BAD
    es = 2
    for call in ("forward", "grad"):
        assert qk(call) == UNSUPPORTED
        assert qk(call, axes=3, sections=(16, 8, 8, 0), ld_positions=6) == UNSUPPORTED
        assert qk(call, axes=3, sections=(32, 0, 0, 9), ld_positions=0) == UNSUPPORTED
        assert qk(call, rotary=0, positions=None, inv_freq=None) == UNSUPPORTED
        # parts of one buffer (768 columns a token), head before token, element alignment
        assert qk(call, q=(P[0], 768, 128), k=(P[0] + 512 * es, 768, 128)) == UNSUPPORTED
        assert qk(call, q_out=(P[6], 768, 128), k_out=(P[6] + 512 * es, 768, 128)) == UNSUPPORTED
        assert qk(call, q_out=(P[6], 128, 6 * 128), k_out=(P[7] + es, 128, 6 * 128)) == UNSUPPORTED
        assert qk(call, k=(P[1], 128, 0)) == UNSUPPORTED               # one head, read twice
        assert qk(call, tokens=1, q_out=(P[6], 0, 128)) == UNSUPPORTED
        for kw in (dict(tokens=-1), dict(tokens=nsmi.NS_MAX_ROWS + 1), dict(q_heads=0), dict(k_heads=0),
                   dict(q_heads=nsmi.NS_MAX_HEADS + 1), dict(dim=0), dict(dim=2), dict(dim=130), dict(dim=260),
                   dict(rotary=-4), dict(rotary=132), dict(rotary=62), dict(axes=0), dict(axes=5),
                   dict(axes=2, sections=(16, 15, 0, 0)), dict(axes=2, sections=(40, -8, 0, 0)),
                   dict(axes=2, sections=(1 << 60, 32, 0, 0)), dict(axes=2, sections=(16, 16, 0, 0), ld_positions=-1),
                   dict(dtype=E4M3), dict(weight_dtype=F16), dict(position_type=3), dict(eps=-1.0), dict(eps=NAN),
                   dict(q_weight=None), dict(k_weight=None), dict(q=(None, 512, 128)), dict(q=(P[0] + 1, 512, 128)),
                   dict(q=(P[0], -1, 128)), dict(k=(P[1], 256, 1 << 40)), dict(positions=None),
                   dict(inv_freq=None), dict(positions=P[4] + 4), dict(inv_freq=P[5] + 2), dict(q_weight=P[2] + 2),
                   dict(q_out=(None, 512, 128)), dict(q_out=(P[6], 511, 128)), dict(q_out=(P[6], 512, 127)),
                   dict(q_out=(P[6], 0, 128)), dict(k_out=(P[6] + 512, 256, 128)), dict(q_out=(P[2], 512, 128)),
                   dict(k_out=(P[4], 256, 128)), dict(k_out=(P[5], 256, 128)), dict(q_out=(P[1], 512, 128)),
                   dict(k_out=(P[0], 256, 128)), dict(q_out=(P[0] + 256, 512, 128)),
                   dict(q_out=(P[6], 700, 128), k_out=(P[6] + 512 * es, 700, 128))):
            assert qk(call, **kw) == BAD, (call, kw)
    assert qk(q_out=(P[0], 512, 128), k_out=(P[1], 256, 128)) == UNSUPPORTED           # in place
    assert qk(tokens=0) == nsmi.NS_OK
    assert qk("grad", q_out=(P[8], 512, 128), k_out=(P[9], 256, 128)) == UNSUPPORTED   # over the gradients
    assert qk("grad", tokens=0) == UNSUPPORTED                                         # weights' zeros are written
    assert qk("grad", tokens=0, dqw=None, dkw=None) == nsmi.NS_OK
    assert qk("grad", q_weight=None, k_weight=None, dqw=None, dkw=None, ws=None, n=0,
              q=(None, 0, 0), k=(None, 0, 0)) == UNSUPPORTED
    assert qk("grad", dqw=None, dkw=None) == UNSUPPORTED
    for kw in (dict(q_weight=None, k_weight=None), dict(dw=E4M3), dict(dqw=P[14] + 2), dict(dqw=P[15] + 4),
               dict(dqw=P[0]), dict(dkw=P[2]), dict(ws=P[8]), dict(ws=P[6]), dict(ws=P[14]),
               dict(q_out=(P[8] + 64, 512, 128)), dict(q_out=(P[9], 512, 128)), dict(q_out=(P[0], 512, 128)),
               dict(k_out=(P[1], 256, 128)), dict(dq_out=(P[8] + 1, 512, 128)), dict(dk_out=(None, 256, 128))):
        assert qk("grad", **kw) == BAD, kw
    for kw in (dict(ws=None), dict(n=255), dict(ws=P[16] + 16)):
        assert qk("grad", **kw) == WS, kw


def attn(call="forward", out=None, lse=P[4], dout=None, dq=None, dk=None, dv=None, ws=P[10], n=64 * MB, **kw):
    a = dict(q=(P[0], 256, 64), k=(P[1], 128, 64), v=(P[2], 128, 64), offsets=P[3], tokens=30, sequences=3, q_heads=4,
             k_heads=2, dim=64, dtype=BF16, clear_rest=0, scale=0.125)
    a.update(kw)
    args = ctypes.byref(heads._AttentionArgs(**a))
    out = part(*(out or (P[5], 256, 64)))
    if call == "forward":
        return nsmi.library().ns_attention(args, out, lse, ws, n, None)
    dout = part(*(dout or (P[6], 256, 64)))
    dq, dk, dv = part(*(dq or (P[7], 256, 64))), part(*(dk or (P[8], 128, 64))), part(*(dv or (P[9], 128, 64)))
    return nsmi.library().ns_attention_grad(args, dout, out, lse, dq, dk, dv, ws, n, None)


def test_attention_refusals():
    lib = nsmi.library()
    one = part(P[0], 256, 64)
    assert lib.ns_attention(None, one, P[1], P[2], MB, None) == BAD
    assert lib.ns_attention_grad(None, one, one, P[1], one, one, one, P[2], MB, None) == BAD
    es = 2
    for call in ("forward", "grad"):
        assert attn(call) == UNSUPPORTED
        assert attn(call, tokens=0, q=(None, 0, 0), k=(None, 0, 0), v=(None, 0, 0), offsets=None) == nsmi.NS_OK
        assert attn(call, dtype=F16, dim=8, sequences=0, clear_rest=1) == UNSUPPORTED
        assert attn(call, q=(P[0], 512, 64), k=(P[0] + 256 * es, 512, 64), v=(P[0] + 384 * es, 512, 64)) == UNSUPPORTED
        assert attn(call, k=(P[1], 64, 0), v=(P[2], 64, 0)) == UNSUPPORTED             # one head, read twice
        assert attn(call, q=(P[0], 64, 30 * 64), out=(P[5], 64, 30 * 64)) == UNSUPPORTED
        assert attn(call, tokens=1, q=(P[0], 3, 64)) == UNSUPPORTED                    # the stride does not count
        for kw in (dict(dtype=F32), dict(dtype=E4M3), dict(tokens=-1), dict(tokens=nsmi.NS_MAX_ROWS + 1),
                   dict(sequences=-1), dict(sequences=nsmi.NS_MAX_ROWS + 1), dict(q_heads=0), dict(k_heads=0),
                   dict(q_heads=5), dict(q_heads=2, k_heads=4), dict(q_heads=2048), dict(dim=0), dict(dim=60),
                   dict(dim=136), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF),
                   dict(offsets=None), dict(offsets=P[3] + 2), dict(lse=None), dict(lse=P[4] + 2),
                   dict(q=(None, 256, 64)), dict(q=(P[0] + 8, 256, 64)), dict(k=(P[1], 124, 64)),
                   dict(k=(P[1], 56, 64)), dict(v=(P[2], 128, 60)), dict(q=(P[0], (1 << 23) + 8, 64)),
                   dict(out=(None, 256, 64)), dict(out=(P[5] + 8, 256, 64)), dict(out=(P[5], 252, 64)),
                   dict(tokens=nsmi.NS_MAX_ROWS, q_heads=1024, k_heads=1024)):
            assert attn(call, **kw) == BAD, (call, kw)
    for kw in (dict(out=(P[5], 248, 64)), dict(out=(P[5], 256, 56)), dict(out=(P[0], 256, 64)), dict(out=(P[1], 256, 64)),
               dict(out=(P[2], 256, 64)), dict(out=(P[3], 256, 64)), dict(out=(P[4], 256, 64)), dict(lse=P[0]),
               dict(lse=P[3]), dict(lse=P[2] + 16)):
        assert attn(**kw) == BAD, kw
    assert attn("grad", dq=(P[7], 512, 64), dk=(P[7] + 256 * es, 512, 64), dv=(P[7] + 384 * es, 512, 64)) == UNSUPPORTED
    for kw in (dict(dq=(P[7], 512, 64), dk=(P[7] + 248 * es, 512, 64)), dict(dq=(P[0], 256, 64)), dict(dk=(P[9], 128, 64)),
               dict(dv=(P[2], 128, 64)), dict(dq=(P[6], 256, 64)), dict(dk=(P[5], 128, 64)), dict(dv=(P[4], 128, 64)),
               dict(dq=(P[3], 256, 64)), dict(dq=(P[7], 256, 32)), dict(dk=(P[8] + 8, 128, 64)), dict(dv=(None, 128, 64)),
               dict(dout=(None, 256, 64)), dict(dout=(P[6] + 8, 256, 64)), dict(ws=P[0]), dict(ws=P[4]), dict(ws=P[7])):
        assert attn("grad", **kw) == BAD, kw
    for kw in (dict(ws=None), dict(n=64), dict(ws=P[10] + 16)):
        assert attn("grad", **kw) == WS, kw
    # nothing is needed for short sequences; for few long ones it is, and checked
    assert attn(ws=None, n=0) == UNSUPPORTED
    long = dict(tokens=5000, sequences=1)
    need = nsmi.ns_attention_workspace_size(5000, 1, 4, 2, 64)
    assert need > 0 and attn(n=need, **long) == UNSUPPORTED
    assert attn(n=need - 1, **long) == WS and attn(ws=None, **long) == WS and attn(ws=P[10] + 64, **long) == WS
    assert attn(ws=P[5], **long) == BAD and attn(ws=P[0], **long) == BAD and attn(ws=P[3], **long) == BAD


def test_workspace_sizes():
    size = nsmi.ns_token_logps_workspace_size
    assert size(0, 1) == 0 and size(4, 1 << 17, 64) > 0 and size(1 << 23, 1 << 23, 64) == 0
    for bad in ((-1, 8, 0), (8, 0, 0), (8, 8, 9), (8, 100, 65), (8, 8, -1), ((1 << 23) + 1, 8, 0)):
        with pytest.raises(nsmi.NsError):
            size(*bad)
    assert nsmi.ns_qk_norm_rope_grad_workspace_size(0, 8) > 0
    for bad in ((-1, 8), (8, 0), (8, 6), (8, 260)):
        with pytest.raises(nsmi.NsError):
            nsmi.ns_qk_norm_rope_grad_workspace_size(*bad)
    for size in (nsmi.ns_attention_workspace_size, nsmi.ns_attention_grad_workspace_size):
        assert size(0, 0, 1, 1, 8) >= 0 and size(1 << 23, 1, 4, 4, 128) >= 0
        for bad in ((-1, 0, 1, 1, 8), (8, -1, 1, 1, 8), (8, 1, 0, 1, 8), (8, 1, 3, 2, 8), (8, 1, 1, 2, 8),
                    (8, 1, 1, 1, 12), (8, 1, 1, 1, 136), (8, 1, 2048, 1, 8)):
            with pytest.raises(nsmi.NsError):
                size(*bad)


def test_python_refusals():
    """What the binding refuses before it has pointers to pass on."""
    import torch
    x, flat = torch.zeros(4, 2, 8), torch.zeros(4, 8)
    ids, w, freq = torch.zeros(4, dtype=torch.int64), torch.zeros(8), torch.zeros(4)
    ends = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: nsmi.ns_token_logps(flat, ids), lambda: nsmi.ns_token_logps_grad(flat, ids, w, w, w),
                 lambda: nsmi.ns_qk_norm_rope(x, x, w, w, ids, freq), lambda: nsmi.ns_qk_norm_rope(flat, x, w, w, ids, freq),
                 lambda: nsmi.ns_qk_norm_rope_grad(x, x, x, x, w, w, ids, freq),
                 lambda: nsmi.ns_attention(x, x, x, ends), lambda: nsmi.ns_attention(flat, flat, flat, ends),
                 lambda: nsmi.ns_attention_grad(x, x, x, x, x, w, ends)):
        with pytest.raises(ValueError):
            call()
