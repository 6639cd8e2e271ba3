"""RMS norm (with the residual's addition, with e4m3 output) and its gradient
against the fp64 forms.

Tolerances. Row sums are added by threads (at most 64 terms each), then over
64 lanes and up to 16 waves: fewer than N = 100 roundings on any path, so a sum
is off by at most N half steps of the sum of magnitudes; rstd by half of that
and three roundings; y by three more and its own rounding. A code is off by
half a step of e4m3 (2^-4 of the value, or half of the smallest subnormal
2^-9) of a quotient that is itself off by the errors of y and of the scale.
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
EPS = 1e-5

SHAPES = [(1, 1), (3, 7), (5, 64), (9, 512), (4, 513), (7, 1024), (3, 1025), (130, 2048), (6, 2049),
          (1, 4096), (11, 4097), (5, 8192), (3, 8193), (2, 16384), (2, 16385), (2, 32768), (2, 32769),
          (2, 65536), (3, 50021), (2500, 96)]


def _expected_y(h, w):
    y, rstd = O.rms_norm(f64(h), f64(w), float(np.float32(EPS)))
    return y, rstd, (N / 2 + 3) * U32


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("dtype,hdtype,wdtype,out", [
    (BF, BF, BF, BF), (BF, SF, SF, BF), (HF, HF, SF, SF), (HF, SF, HF, HF), (SF, SF, SF, BF)])
def test_norm(rows, dim, dtype, hdtype, wdtype, out):
    require_gpu()
    print("norm", rows, dim, dtype, hdtype, out, flush=True)
    x, w = normal(rows, (rows, dim), dtype), normal(dim, (dim,), wdtype)
    y, h, rstd = nsmi.ns_rms_norm(x, w, eps=EPS, out_dtype=out)
    assert h is x and y.dtype == out
    want, r, rel = _expected_y(x, w)
    assert_within(rstd, r, rel * r, "rstd")
    slack = (rel + 3 * U32) * np.abs(want) * 1.01
    assert_within(y, want, slack + 1.01 * half_step(np.abs(want) + slack, out), "y")
    res = normal(rows + 1, (rows, dim), hdtype, 3.0)
    y, h, rstd = nsmi.ns_rms_norm(x, w, residual=res, eps=EPS, out_dtype=out)
    # the sum of two values of at most 24 bits rounds once in fp32 and once to h's type
    both = f64(x) + f64(res)
    assert_within(h, both, U32 * np.abs(both) * 1.01 + 1.01 * half_step(both, hdtype), "h")
    assert h.dtype == hdtype
    want, r, rel = _expected_y(h, w)
    assert_within(rstd, r, rel * r, "rstd")
    slack = (rel + 3 * U32) * np.abs(want) * 1.01
    assert_within(y, want, slack + 1.01 * half_step(np.abs(want) + slack, out), "y")


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 33), (4, 512), (5, 1111), (130, 2048), (9, 4096),
                                      (3, 8200), (2, 20000), (2, 65536)])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_norm_to_e4m3(rows, dim, dtype):
    require_gpu()
    print("e4m3", rows, dim, dtype, flush=True)
    x, w = normal(rows, (rows, dim), dtype), normal(dim, (dim,), dtype)
    res = normal(rows + 2, (rows, dim), dtype)
    q, scales, h, rstd = nsmi.ns_rms_norm_fp8(x, w, residual=res, eps=EPS)
    assert q.dtype == torch.float8_e4m3fn and scales.shape == (rows,)
    want, r, rel = _expected_y(h, w)
    rel = rel + 3 * U32
    assert_within(rstd, r, rel * r, "rstd")
    top = np.abs(want).max(-1)
    assert_within(scales, top / 448, (rel + 2 * U32) * top / 448 * 1.01, "scales")
    code = want / (top / 448)[:, None]
    slack = (2 * rel + 6 * U32) * np.abs(code)
    assert_within(q.float(), code, slack + np.maximum((np.abs(code) + slack) * 2.0 ** -4, 2.0 ** -10), "codes")
    assert np.all(np.abs(f64(q.float())).max(-1) == 448)


def test_e4m3_codes_are_torchs():
    """Bit for bit the rounding of torch's own conversion, for every exponent."""
    require_gpu()
    v = torch.linspace(-1, 1, 4096, device="cuda")
    x = torch.stack([v, v ** 3, v ** 9, v.sign() * 2.0 ** (-30 * v.abs())])
    q, scales, _, rstd = nsmi.ns_rms_norm_fp8(x, torch.ones(4096, device="cuda"), eps=0.0)
    y, _, _ = nsmi.ns_rms_norm(x, torch.ones(4096, device="cuda"), eps=0.0)
    want = (y * (1.0 / scales)[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


def test_rows_of_zeros_infinities_and_nan():
    require_gpu()
    for dim in (40, 1000, 4096, 20000):
        x = normal(1, (6, dim), SF)
        x[1] = 0
        x[2, 3], x[3, 5], x[4] = float("inf"), float("nan"), 1e-30
        w = torch.ones(dim, device="cuda")
        y, _, rstd = nsmi.ns_rms_norm(x, w, eps=1e-6)
        assert torch.all(y[1] == 0) and torch.isfinite(y[0]).all()
        assert rstd[2] == 0 and torch.isnan(y[2, 3]) and torch.all(y[2, 4:] == 0)
        assert torch.isnan(y[3]).all() and torch.isfinite(y[4]).all()
        q, scales, _, _ = nsmi.ns_rms_norm_fp8(x, w, eps=1e-6)
        assert scales[1] == 1 and torch.all(q[1].float() == 0)
        assert torch.isnan(q[3].float()).all() and torch.isnan(q[2, 3].float())
        assert torch.isfinite(scales[[0, 1, 2, 4, 5]]).all()
        # a zero row with eps = 0: 0 * inf
        z, _, r0 = nsmi.ns_rms_norm(x, w, eps=0.0)
        assert torch.isinf(r0[1]) and torch.isnan(z[1]).all()


def test_norm_in_place_of_the_residual_and_of_x():
    require_gpu()
    for dim in (5, 96, 1000, 4099, 5000, 20001):
        x, res, w = normal(1, (9, dim), BF), normal(2, (9, dim), BF), normal(3, (dim,), BF)
        y, h, rstd = nsmi.ns_rms_norm(x, w, residual=res)
        for target in ("res", "x"):
            a, b = x.clone(), res.clone()
            t = b if target == "res" else a
            y2, h2, r2 = nsmi.ns_rms_norm(a, w, residual=b, h=t)
            assert h2 is t and torch.equal(h2, h) and torch.equal(y2, y) and torch.equal(r2, rstd)
        wide = res.float()
        _, h3, _ = nsmi.ns_rms_norm(x, w, residual=wide, h=wide)
        assert h3 is wide and torch.equal(wide, x.float() + res.float())


def test_norm_strided_unaligned_and_many_dimensions():
    require_gpu()
    for dtype in (BF, SF):
        x, _ = strided_rows(normal(1, (12, 301), dtype), 7, 1)
        res, _ = strided_rows(normal(2, (12, 301), dtype), 4, 3)
        h, store = strided_rows(torch.zeros(12, 301, dtype=dtype, device="cuda"), 2, 5)
        w = normal(3, (302,), dtype)[1:]
        y, _, rstd = nsmi.ns_rms_norm(x, w, residual=res, h=h)
        y2, h2, r2 = nsmi.ns_rms_norm(x.contiguous(), w.clone(), residual=res.contiguous())
        assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(rstd, r2)
        assert untouched(store, h)
    # heads of a (tokens, heads, dim) tensor inside a wider projection
    qkv = normal(4, (6, 5, 3, 64), BF)
    part = qkv[:, :, 1]
    y, _, rstd = nsmi.ns_rms_norm(part, normal(5, (64,), BF))
    y2, _, _ = nsmi.ns_rms_norm(part.contiguous(), normal(5, (64,), BF))
    assert y.shape == (6, 5, 64) and rstd.shape == (6, 5) and torch.equal(y, y2)


def test_norm_of_no_rows():
    require_gpu()
    x, w = torch.empty((0, 48), dtype=BF, device="cuda"), normal(1, (48,), BF)
    y, h, rstd = nsmi.ns_rms_norm(x, w, residual=x.float())
    assert y.shape == (0, 48) and rstd.shape == (0,)
    assert nsmi.ns_rms_norm_fp8(x, w)[0].shape == (0, 48)
    dx, dw = nsmi.ns_rms_norm_grad(x, x, w, rstd, dweight_dtype=SF)
    assert dx.shape == (0, 48) and torch.all(dw == 0)


def _grad_expected(dy, h, w, rstd, dh):
    """Formula with the rstd given (the kernel takes it as an input), and slacks."""
    dy, h, w, r = f64(dy), f64(h), f64(w), f64(rstd)[:, None]
    u, g = h * r, dy * w
    mean, mag = np.mean(g * u, -1, keepdims=True), np.mean(np.abs(g * u), -1, keepdims=True)
    dx = r * (g - u * mean)
    # g and u are rounded, their product is added up, then three more roundings
    slack = np.abs(r) * (4 * np.abs(g) + np.abs(u) * (5 * np.abs(mean) + (N + 4) * mag)) * U32
    if dh is not None:
        dx = dx + f64(dh)
        slack = slack + U32 * np.abs(dx)
    rows = dy.shape[0]
    dw, dmag = np.sum(dy * u, 0), np.sum(np.abs(dy * u), 0)
    return dx, slack * 1.01, dw, (rows + 70) * U32 * dmag


@pytest.mark.parametrize("rows,dim", SHAPES + [(1031, 1111), (4500, 40)])
@pytest.mark.parametrize("dtype,hdtype,wdtype,dxdtype,dwdtype", [
    (BF, BF, BF, BF, BF), (BF, SF, SF, SF, SF), (HF, HF, HF, SF, SF), (SF, SF, SF, SF, SF)])
def test_gradient(rows, dim, dtype, hdtype, wdtype, dxdtype, dwdtype):
    require_gpu()
    print("norm gradient", rows, dim, dtype, hdtype, dxdtype, flush=True)
    h, w = normal(rows, (rows, dim), hdtype, 2.0), normal(dim, (dim,), wdtype)
    dy = normal(rows + 1, (rows, dim), dtype)
    _, rstd64 = O.rms_norm(f64(h), f64(w), EPS)
    rstd = torch.from_numpy(rstd64).float().cuda()
    for dh in (None, normal(rows + 2, (rows, dim), dxdtype)):
        dx, dw = nsmi.ns_rms_norm_grad(dy, h, w, rstd, dh=dh, dx_dtype=dxdtype, dweight_dtype=dwdtype)
        wx, sx, ww, sw = _grad_expected(dy, h, w, rstd, dh)
        assert dx.dtype == dxdtype and dw.dtype == dwdtype
        assert_within(dx, wx, sx + 1.01 * half_step(np.abs(wx) + sx, dxdtype), "dx")
        assert_within(dw, ww, sw + 1.01 * half_step(np.abs(ww) + sw, dwdtype), "dw")
    dx2, dw2 = nsmi.ns_rms_norm_grad(dy, h, w, rstd, dh=dh, dx=dh, dweight_dtype=dwdtype)   # in place
    assert dx2 is dh and torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_gradient_against_differences():
    """<dx, t> and <dw, s> against central differences of the fp64 forward."""
    require_gpu()
    rows, dim, d = 6, 150, 1e-5
    h, w, dy = normal(1, (rows, dim)), normal(2, (dim,)), normal(3, (rows, dim))
    _, _, rstd = nsmi.ns_rms_norm(h, w, eps=EPS)
    dx, dw = nsmi.ns_rms_norm_grad(dy, h, w, rstd)
    H, W, DY, t, s = f64(h), f64(w), f64(dy), f64(normal(4, (rows, dim))), f64(normal(5, (dim,)))
    f = lambda a, b: np.sum(DY * O.rms_norm(a, b, float(np.float32(EPS)))[0])   # noqa: E731
    # differences are good to 1e-8 here; the kernel's sums to N half steps of their magnitudes
    slope = (f(H + d * t, W) - f(H - d * t, W)) / (2 * d)
    assert abs(slope - np.sum(f64(dx) * t)) <= 1e-6 + 2 * N * U32 * np.sum(np.abs(f64(dx) * t))
    slope = (f(H, W + d * s) - f(H, W - d * s)) / (2 * d)
    assert abs(slope - np.sum(f64(dw) * s)) <= 1e-6 + 2 * N * U32 * np.sum(np.abs(f64(dw) * s))


def test_gradient_strided_and_unaligned():
    require_gpu()
    for dim in (45, 3001):
        dy, _ = strided_rows(normal(1, (12, dim), BF), 3, 1)
        h, _ = strided_rows(normal(2, (12, dim), BF), 2, 5)
        dh, _ = strided_rows(normal(3, (12, dim), BF), 6, 3)
        dx, store = strided_rows(torch.zeros(12, dim, dtype=BF, device="cuda"), 1, 7)
        w = normal(4, (dim,), BF)
        _, _, rstd = nsmi.ns_rms_norm(h, w)
        _, dw = nsmi.ns_rms_norm_grad(dy, h, w, rstd, dh=dh, dx=dx)
        dx2, dw2 = nsmi.ns_rms_norm_grad(dy.contiguous(), h.contiguous(), w, rstd, dh=dh.contiguous())
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        assert untouched(store, dx)


def test_offsets_beyond_32_bits():
    require_gpu()
    rows, dim = 40000, 65536
    x = torch.zeros((rows, dim), dtype=BF, device="cuda")
    x[-1], x[-2, 0] = 2.0, 1.0
    w = torch.ones(dim, dtype=BF, device="cuda")
    y, _, rstd = nsmi.ns_rms_norm(x, w, eps=0.25)
    assert abs(rstd[-1].item() - 4.25 ** -0.5) < 1e-6 and torch.all(rstd[:-2] == 2.0)
    assert y[-1].float().mean().item() == torch.tensor(2 * 4.25 ** -0.5).to(BF).item()
    dx, dw = nsmi.ns_rms_norm_grad(x, x, w, rstd, dx=y, dweight_dtype=SF)
    assert torch.all(dx[:-2] == 0) and dx[-1].float().abs().max() > 0
    assert torch.all(torch.isfinite(dw)) and dw[5].item() == pytest.approx(4 * 4.25 ** -0.5, rel=1e-5)
