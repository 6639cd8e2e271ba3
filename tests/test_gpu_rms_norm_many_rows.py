"""RMS norm and its gradient where a workgroup takes several rows, for each
team size, and where an output of 2^23 elements or more leaves past the caches.

A workgroup of the forward kernel takes further rows above 8192 rows (up to
1024 columns), 2048 (up to 2048), 1024 (up to 4096), 1364 (up to 6144) and 1024
(up to 8192); one of the gradient above 4096, 1024, 512, 341 and 256 rows.
Tolerances: fewer than N = 100 roundings on any path of a row's sum, so rstd is
off by N / 2 + 3 half steps and y by three more and its own rounding; a code by
half a step of e4m3 of a quotient off by the errors of y and of its scale.
"""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import train_oracle as O
from train_helpers import U32, assert_within, f64, half_step, normal, strided_rows, untouched

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
N = 100
EPS = float(np.float32(1e-5))
REL = (N / 2 + 3) * U32

LOOPS = [(8200, 512), (8300, 100), (8195, 700), (8200, 1024), (2100, 1111), (2060, 2048), (1100, 4096),
         (1030, 2500), (1400, 5001), (1370, 6144), (1100, 8191), (1030, 8192)]
STREAMED = [(16500, 513), (8200, 1024), (4200, 2048), (2100, 4096), (2100, 3997), (1700, 5001),
            (1030, 8192), (1100, 8191)]


def _check_norm(x, res, w, out, h_in_place):
    """One call against the oracle; returns its outputs."""
    hdtype = res.dtype
    both = f64(x) + f64(res)
    into = res.clone()
    if out == "e4m3":
        y, scales, h, rstd = nsmi.ns_rms_norm_fp8(x, w, residual=into, eps=EPS, h=into if h_in_place else None)
    else:
        y, h, rstd = nsmi.ns_rms_norm(x, w, residual=into, eps=EPS, out_dtype=out, h=into if h_in_place else None)
    assert (h is into) == h_in_place and (h_in_place or torch.equal(into, res))
    assert_within(h, both, U32 * np.abs(both) * 1.01 + 1.01 * half_step(both, hdtype), "h")
    want, r = O.rms_norm(f64(h), f64(w), EPS)
    assert_within(rstd, r, REL * r, "rstd")
    if out != "e4m3":
        slack = (REL + 3 * U32) * np.abs(want) * 1.01
        assert_within(y, want, slack + 1.01 * half_step(np.abs(want) + slack, out), "y")
        return y, h, rstd
    rel = REL + 3 * U32
    top = np.abs(want).max(-1) / 448
    assert_within(scales, top, (rel + 2 * U32) * top * 1.01, "scales")
    code = np.abs(want / top[:, None])
    slack = (2 * rel + 6 * U32) * code
    assert_within(y.float(), want / top[:, None],
                  slack + np.maximum((code + slack) * 2.0 ** -4, 2.0 ** -10), "codes")
    return y.view(torch.uint8), scales, h, rstd


@pytest.mark.parametrize("rows,dim", LOOPS)
@pytest.mark.parametrize("dtype,hdtype,out", [(BF, BF, BF), (HF, SF, "e4m3"), (SF, SF, HF)])
def test_rows_in_turn(rows, dim, dtype, hdtype, out):
    require_gpu()
    print("rows in turn", rows, dim, dtype, hdtype, out, flush=True)
    x, w = normal(rows, (rows, dim), dtype), normal(dim, (dim,), dtype)
    _check_norm(x, normal(rows + 1, (rows, dim), hdtype, 3.0), w, out, False)


@pytest.mark.parametrize("rows,dim", STREAMED)
@pytest.mark.parametrize("out", [BF, "e4m3"])
def test_large_outputs(rows, dim, out):
    """Past 2^23 elements: y, or beside codes h, leaves past the caches."""
    require_gpu()
    print("large outputs", rows, dim, out, flush=True)
    assert rows * dim >= 1 << 23
    x, w = normal(rows, (rows, dim), BF), normal(dim, (dim,), BF)
    res = normal(rows + 1, (rows, dim), BF, 3.0)
    apart = _check_norm(x, res, w, out, False)
    same = _check_norm(x, res, w, out, True)
    assert all(torch.equal(a, b) for a, b in zip(apart, same)), "h in the residual's place"
    # the same rows a thousand at a time, below the limit: the same bits
    part = slice(0, 1000)
    few = _check_norm(x[part], res[part], w, out, False)
    assert all(torch.equal(a[part], b) for a, b in zip(apart, few))


def test_large_outputs_in_strided_rows():
    """What lies between the rows of h is not written; x in fp16, y too."""
    require_gpu()
    rows, dim = 2100, 4001
    x, w = normal(1, (rows, dim), HF), normal(2, (dim,), HF)
    res, _ = strided_rows(normal(3, (rows, dim), HF, 3.0), 7, 1)
    h, store = strided_rows(torch.zeros(rows, dim, dtype=HF, device="cuda"), 5, 3)
    want = nsmi.ns_rms_norm(x, w, residual=res.contiguous(), eps=EPS)
    y, _, rstd = nsmi.ns_rms_norm(x, w, residual=res, eps=EPS, h=h)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and torch.equal(rstd, want[2])
    q, scales, _, _ = nsmi.ns_rms_norm_fp8(x, w, residual=res, eps=EPS, h=h)
    q2, scales2, _, _ = nsmi.ns_rms_norm_fp8(x, w, residual=res.contiguous(), eps=EPS)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scales, scales2)
    assert torch.equal(h, want[1]) and untouched(store, h)


@pytest.mark.parametrize("rows,dim", [(4500, 513), (4500, 1024), (1100, 1111), (600, 4096), (550, 2049),
                                      (400, 5001), (400, 6144), (300, 8191), (300, 8192)])
@pytest.mark.parametrize("dtype,hdtype,dxdtype", [(BF, BF, BF), (HF, SF, SF), (SF, SF, SF)])
def test_gradient_rows_in_turn(rows, dim, dtype, hdtype, dxdtype):
    """dx: g and u are rounded, their product added up, three more roundings.
    dw: a rounding of u and one at each row of a workgroup's share (the rows
    of the whole call at most), of teams' shares at four more."""
    require_gpu()
    print("gradient rows in turn", rows, dim, dtype, hdtype, dxdtype, flush=True)
    h, w = normal(rows, (rows, dim), hdtype, 2.0), normal(dim, (dim,), dtype)
    dy, dh = normal(rows + 1, (rows, dim), dtype), normal(rows + 2, (rows, dim), dxdtype)
    rstd = torch.from_numpy(O.rms_norm(f64(h), f64(w), EPS)[1]).float().cuda()
    dx, dw = nsmi.ns_rms_norm_grad(dy, h, w, rstd, dh=dh, dx_dtype=dxdtype, dweight_dtype=SF)
    DY, W, r = f64(dy), f64(w), f64(rstd)[:, None]
    u, g = f64(h) * r, DY * W
    mean, mag = np.mean(g * u, -1, keepdims=True), np.mean(np.abs(g * u), -1, keepdims=True)
    want = r * (g - u * mean) + f64(dh)
    slack = np.abs(r) * (4 * np.abs(g) + np.abs(u) * (5 * np.abs(mean) + (N + 4) * mag)) * U32
    slack = (slack + U32 * np.abs(want)) * 1.01
    assert_within(dx, want, slack + 1.01 * half_step(np.abs(want) + slack, dxdtype), "dx")
    sums, mags = np.sum(DY * u, 0), np.sum(np.abs(DY * u), 0)
    assert_within(dw, sums, ((rows + 6) * U32 * mags + U32 * np.abs(sums)) * 1.01, "dw")
    dx2, dw2 = nsmi.ns_rms_norm_grad(dy, h, w, rstd, dh=dh, dx=dh, dweight_dtype=SF)     # in place
    assert dx2 is dh and torch.equal(dx2, dx) and torch.equal(dw2, dw)
