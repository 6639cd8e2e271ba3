"""Refusals of the operators around the matrix update, at the C ABI, without a
GPU: bad arguments are answered before any device work (the addresses here
belong to nothing and are never touched), and valid ones reach the device
check."""

import ctypes

import pytest

import newton_schulz_matrix_amd as nsmi
from newton_schulz_matrix_amd import operators as ops

import os

pytestmark = pytest.mark.skipif(not os.path.exists(nsmi.LIB_PATH), reason="libnsmi.so not built")

BAD, UNSUPPORTED, WS = nsmi.NS_ERR_INVALID_ARG, nsmi.NS_ERR_UNSUPPORTED, nsmi.NS_ERR_WORKSPACE
F32, BF16, F16, E4M3 = nsmi.NS_DT_F32, nsmi.NS_DT_BF16, nsmi.NS_DT_F16, nsmi.NS_DT_E4M3
MB = 1 << 20
# addresses 64 MB apart
P = [(64 + 64 * i) * MB for i in range(16)]


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")


def lookup(**kw):
    a = dict(table=P[0], dt=BF16, rows=10, dim=64, ld=64, ids=P[1], idt=1, count=5, scale=1.0,
             out=P[2], odt=BF16, ldo=64)
    a.update(kw)
    return nsmi.library().ns_embedding(*a.values(), None)


def test_embedding_refusals():
    assert lookup() == UNSUPPORTED       # valid, but there is no device
    assert lookup(count=0, ids=None, out=None) == nsmi.NS_OK
    for kw in (dict(table=None), dict(ids=None), dict(out=None), dict(dt=3), dict(dt=7), dict(odt=3),
               dict(idt=2), dict(rows=0), dict(rows=nsmi.NS_MAX_ROWS + 1), dict(dim=0),
               dict(dim=65537, ld=65537, ldo=65537), dict(ld=63), dict(ldo=63), dict(count=-1),
               dict(count=nsmi.NS_MAX_ROWS + 1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(table=P[0] + 1), dict(ids=P[1] + 4), dict(out=P[2] + 1), dict(ld=1 << 40),
               dict(out=P[0] + 128), dict(out=P[1] + 8)):
        assert lookup(**kw) == BAD, kw
    assert lookup(ids=P[1] + 4, idt=0) == UNSUPPORTED
    assert lookup(table=P[0] + 2, out=P[2] + 6) == UNSUPPORTED     # element alignment is enough
    assert lookup(out=P[0] + 10 * 128) == UNSUPPORTED              # right behind the table


def emb_grad(**kw):
    a = dict(g=P[0], gdt=BF16, ldg=64, ids=P[1], idt=1, count=500, rows=10, dim=64, scale=1.0, pad=-1,
             acc=0, out=P[2], odt=F32, ldo=64, ws=P[3], n=64 * MB)
    a.update(kw)
    return nsmi.library().ns_embedding_grad(*a.values(), None)


def test_embedding_grad_refusals():
    assert emb_grad() == UNSUPPORTED
    assert emb_grad(count=0, g=None, ids=None) == UNSUPPORTED      # zeros are written
    assert emb_grad(count=0, g=None, ids=None, acc=1, ws=None, n=0) == nsmi.NS_OK
    assert emb_grad(pad=3) == UNSUPPORTED
    for kw in (dict(g=None), dict(ids=None), dict(out=None), dict(gdt=3), dict(odt=9), dict(idt=-1),
               dict(rows=0), dict(dim=0), dict(count=-1), dict(ldg=60), dict(ldo=1),
               dict(scale=float("nan")), dict(g=P[0] + 1), dict(out=P[2] + 2), dict(ids=P[1] + 2),
               dict(out=P[0]), dict(out=P[1] + 800), dict(ws=P[2]), dict(ws=P[0])):
        assert emb_grad(**kw) == BAD, kw
    need = nsmi.ns_embedding_grad_workspace_size(10, 64, 500)
    assert emb_grad(n=need) == UNSUPPORTED
    for kw in (dict(ws=None, n=0), dict(n=need - 1), dict(ws=P[3] + 16)):
        assert emb_grad(**kw) == WS, kw


def test_workspace_sizes():
    size = nsmi.ns_embedding_grad_workspace_size
    assert size(1, 1, 0) > 0 and size(1 << 23, 65536, 1 << 23) > size(1 << 23, 1, 1 << 23)
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, -1), ((1 << 23) + 1, 8, 8), (8, 8, (1 << 23) + 1)):
        with pytest.raises(nsmi.NsError):
            size(*bad)
    assert nsmi.ns_rms_norm_grad_workspace_size(0, 8) > 0
    for bad in ((-1, 8), (8, 0), (8, 65537)):
        with pytest.raises(nsmi.NsError):
            nsmi.ns_rms_norm_grad_workspace_size(*bad)
    size = nsmi.ns_preference_loss_workspace_size
    assert size(0, 0, 1) > 0 and size(1 << 11, 1 << 11, 1 << 23) > 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), (1 << 12, 1 << 11, 8), (1 << 23, 1, 8)):
        with pytest.raises(nsmi.NsError):
            size(*bad)


def norm(**kw):
    a = dict(x=P[0], residual=P[1], h=P[2], weight=P[3], y=P[4], scales=None, rstd=P[5], rows=8,
             dim=64, ldx=64, ld_residual=64, ldh=64, ldy=64, x_dtype=BF16, h_dtype=BF16,
             weight_dtype=BF16, y_dtype=BF16, eps=1e-6)
    a.update(kw)
    return nsmi.library().ns_rms_norm(ctypes.byref(ops._RmsNormArgs(**a)), None)


def test_rms_norm_refusals():
    assert nsmi.library().ns_rms_norm(None, None) == BAD
    assert norm() == UNSUPPORTED
    assert norm(residual=None, h=None) == UNSUPPORTED
    assert norm(h_dtype=F32, weight_dtype=F32, y_dtype=F16, rstd=None) == UNSUPPORTED
    assert norm(y_dtype=E4M3, scales=P[6]) == UNSUPPORTED
    assert norm(y_dtype=E4M3, scales=P[6], y=P[4] + 3, ldy=65) == UNSUPPORTED
    assert norm(h=P[1]) == UNSUPPORTED and norm(h=P[0]) == UNSUPPORTED       # in place
    assert norm(rows=0, x=None, residual=None, h=None, y=None, h_dtype=F32) == nsmi.NS_OK
    for kw in (dict(x=None), dict(weight=None), dict(y=None), dict(residual=None), dict(h=None),
               dict(residual=None, h=None, h_dtype=F32), dict(scales=P[6]), dict(y_dtype=E4M3),
               dict(x_dtype=E4M3), dict(x_dtype=4), dict(h_dtype=F16), dict(weight_dtype=F16),
               dict(y_dtype=5), dict(rows=-1), dict(rows=nsmi.NS_MAX_ROWS + 1), dict(dim=0),
               dict(dim=70000, ldx=70000, ldh=70000, ldy=70000, ld_residual=70000), dict(ldx=63),
               dict(ldh=1), dict(ldy=0), dict(ld_residual=63), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=P[0] + 1), dict(rstd=P[5] + 2), dict(h=P[2] + 1),
               dict(y=P[0]), dict(y=P[1]), dict(y=P[2] + 64), dict(y=P[3]), dict(rstd=P[4]),
               dict(h=P[1] + 2), dict(h=P[1], ldh=72), dict(h=P[0], h_dtype=F32, ldh=64),
               dict(h=P[3]), dict(rstd=P[3])):
        assert norm(**kw) == BAD, kw


def norm_grad(ws=P[9], n=64 * MB, **kw):
    a = dict(dy=P[0], h=P[1], weight=P[2], rstd=P[3], dh=P[4], dx=P[5], dweight=P[6], rows=8, dim=64,
             lddy=64, ldh=64, lddh=64, lddx=64, dy_dtype=BF16, h_dtype=BF16, weight_dtype=BF16,
             dx_dtype=BF16, dweight_dtype=F32)
    a.update(kw)
    return nsmi.library().ns_rms_norm_grad(ctypes.byref(ops._RmsNormGradArgs(**a)), ws, n, None)


def test_rms_norm_grad_refusals():
    assert nsmi.library().ns_rms_norm_grad(None, P[9], 64 * MB, None) == BAD
    assert norm_grad() == UNSUPPORTED
    assert norm_grad(dh=None, dweight=None, lddh=0) == UNSUPPORTED
    assert norm_grad(dh=P[5]) == UNSUPPORTED                                   # in place
    assert norm_grad(rows=0, dy=None, h=None, dx=None, rstd=None, dweight=None) == nsmi.NS_OK
    for kw in (dict(dy=None), dict(h=None), dict(weight=None), dict(rstd=None), dict(dx=None),
               dict(dy_dtype=E4M3), dict(h_dtype=F16), dict(weight_dtype=F16), dict(dx_dtype=F16),
               dict(dweight_dtype=3), dict(rows=-1), dict(dim=0), dict(lddy=63), dict(ldh=63),
               dict(lddh=63), dict(lddx=63), dict(dx=P[0]), dict(dx=P[1]), dict(dx=P[4] + 2),
               dict(dh=P[5], lddx=72), dict(dweight=P[2]), dict(dweight=P[5] + 4), dict(ws=P[0]),
               dict(ws=P[5]), dict(rstd=P[3] + 1), dict(dweight=P[6] + 2)):
        assert norm_grad(**kw) == BAD, kw
    for kw in (dict(ws=None), dict(n=0), dict(ws=P[9] + 64)):
        assert norm_grad(**kw) == WS, kw


def pref(call="loss", ws=P[8], n=64 * MB, ref=P[2], losses=P[3], margins=P[4], logps=P[5], lse=P[6],
         dlosses=P[3], out=P[7], ld_out=100, **kw):
    a = dict(logits=P[0], labels=P[1], pairs=2, length=3, vocab=100, ld=100, dtype=BF16, label_type=1,
             beta=0.1, label_smoothing=0.0, ld_sequence=0)
    a.update(kw)
    args = ctypes.byref(ops._PreferenceArgs(*a.values()))
    if call == "loss":
        return nsmi.library().ns_preference_loss(args, ref, losses, margins, logps, lse, ws, n, None)
    return nsmi.library().ns_preference_loss_grad(args, margins, lse, dlosses, out, ld_out, None)


def test_preference_refusals():
    lib = nsmi.library()
    assert lib.ns_preference_loss(None, *P[2:7], P[8], MB, None) == BAD
    assert lib.ns_preference_loss_grad(None, *P[2:5], P[7], 100, None) == BAD
    for call in ("loss", "grad"):
        assert pref(call) == UNSUPPORTED
        assert pref(call, pairs=0, logits=None, labels=None) == nsmi.NS_OK
        for kw in (dict(logits=None), dict(labels=None), dict(margins=None), dict(lse=None),
                   dict(pairs=-1), dict(length=-1), dict(vocab=0), dict(ld=99), dict(dtype=3),
                   dict(label_type=2), dict(beta=float("inf")), dict(label_smoothing=-0.1),
                   dict(label_smoothing=1.1), dict(label_smoothing=float("nan")),
                   dict(pairs=1 << 12, length=1 << 11), dict(vocab=nsmi.NS_MAX_ROWS + 1, ld=1 << 30),
                   dict(logits=P[0] + 1), dict(labels=P[1] + 4), dict(margins=P[4] + 2)):
            assert pref(call, **kw) == BAD, (call, kw)
    for kw in (dict(ref=None), dict(losses=None), dict(logps=None), dict(losses=P[4]), dict(lse=P[0]),
               dict(logps=P[2]), dict(ws=P[0]), dict(ws=P[6])):
        assert pref(**kw) == BAD, kw
    for kw in (dict(ws=None), dict(n=8), dict(ws=P[8] + 8)):
        assert pref(**kw) == WS, kw
    assert pref("grad", out=P[0]) == UNSUPPORTED                               # in place
    for call in ("loss", "grad"):
        assert pref(call, ld_sequence=400) == UNSUPPORTED and pref(call, ld_sequence=300) == UNSUPPORTED
        for bad in (299, 1, -5, 1 << 60):
            assert pref(call, ld_sequence=bad) == BAD, bad
    assert pref("grad", ld_sequence=MB, out=P[0] + 8 * MB) == UNSUPPORTED      # behind 4 sequences
    assert pref("grad", ld_sequence=MB, out=P[0] + 3 * MB) == BAD
    assert pref("grad", length=0, logits=None, labels=None, out=None) == nsmi.NS_OK
    for kw in (dict(out=None), dict(dlosses=None), dict(ld_out=99), dict(out=P[0], ld_out=104),
               dict(out=P[0] + 2), dict(out=P[1]), dict(out=P[4]), dict(out=P[6]), dict(out=P[7] + 1)):
        assert pref("grad", **kw) == BAD, kw


def adamw(step=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, count=1, **kw):
    a = dict(param=P[0], grad=P[1], exp_avg=P[2], exp_avg_sq=P[3], master=P[4], elems=1000,
             param_dtype=BF16, grad_dtype=F16, exp_avg_dtype=F32, exp_avg_sq_dtype=F32,
             weight_decay=0.1)
    a.update(kw)
    t = (ops._AdamwTensor * 1)(ops._AdamwTensor(*a.values()))
    return nsmi.library().ns_adamw_step(t, count, step, lr, beta1, beta2, eps, None)


def test_adamw_refusals():
    nan, inf = float("nan"), float("inf")
    assert adamw() == UNSUPPORTED and adamw(master=None) == UNSUPPORTED
    assert adamw(count=0) == nsmi.NS_OK
    assert adamw(elems=0, param=None, grad=None) == nsmi.NS_OK
    assert nsmi.library().ns_adamw_step(None, 1, 1, 0.1, 0.9, 0.9, 0.1, None) == BAD
    for kw in (dict(count=-1), dict(step=0), dict(step=-3), dict(lr=-0.1), dict(lr=nan), dict(lr=inf),
               dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=nan), dict(eps=-1e-9),
               dict(eps=inf), dict(param=None), dict(grad=None), dict(exp_avg=None),
               dict(exp_avg_sq=None), dict(elems=-1), dict(elems=(1 << 33) + 1), dict(param_dtype=3),
               dict(grad_dtype=4), dict(exp_avg_dtype=-1), dict(exp_avg_sq_dtype=F16),
               dict(weight_decay=-0.1), dict(weight_decay=nan), dict(param=P[0] + 1),
               dict(exp_avg=P[2] + 2), dict(master=P[4] + 2), dict(grad=P[0]), dict(exp_avg=P[3] + 400),
               dict(master=P[0])):
        assert adamw(**kw) == BAD, kw


def test_python_refusals():
    """What the binding refuses before it has pointers to pass on."""
    import torch
    cpu = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: nsmi.ns_embedding(cpu, ids), lambda: nsmi.ns_embedding(cpu[0], ids),
                 lambda: nsmi.ns_embedding_grad(cpu, ids, 4), lambda: nsmi.ns_rms_norm(cpu, cpu[0]),
                 lambda: nsmi.ns_rms_norm_fp8(cpu, cpu[0]),
                 lambda: nsmi.ns_rms_norm_grad(cpu, cpu, cpu[0], cpu[:, 0]),
                 lambda: nsmi.ns_preference_loss(cpu, ids, cpu[0]),
                 lambda: nsmi.ns_preference_loss(cpu[None].expand(3, 4, 8), ids, cpu[0]),
                 lambda: nsmi.ns_adamw_step([cpu], [cpu], [cpu], [cpu], 1, 0.1),
                 lambda: nsmi.ns_adamw_step([cpu], [cpu], [cpu], [], 1, 0.1)):
        with pytest.raises(ValueError):
            call()
    assert nsmi.ns_adamw_step([], [], [], [], 1, 0.1) is None
