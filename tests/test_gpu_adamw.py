"""AdamW step against the fp64 form.

Tolerances. m and v are each two products and a sum (three roundings of the
terms' magnitudes, plus the rounding of the constants) and one rounding to
their type. The update is taken from unrounded m and v: m's error, half of
v's, and eight roundings of its own, relative; then two roundings of w, and
one to the parameter's type.
"""

import numpy as np
import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from oracle import train_oracle as O
from train_helpers import U32, assert_within, f64, half_step, normal

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
LR, BETAS, EPS = 2e-3, (0.9, 0.999), 1e-8


def _state(seed, shape, p, g, m, v, master):
    w = normal(seed, shape, SF)
    return dict(param=w.to(p, copy=True), master=w if master else None, grad=normal(seed + 1, shape, g, 0.1),
                exp_avg=normal(seed + 2, shape, m, 0.05),
                exp_avg_sq=normal(seed + 3, shape, SF, 0.1).square().to(v))


def _step(states, step, decays, betas=BETAS, eps=EPS, lr=LR):
    nsmi.ns_adamw_step([s["param"] for s in states], [s["grad"] for s in states],
                       [s["exp_avg"] for s in states], [s["exp_avg_sq"] for s in states], step=step,
                       lr=lr, betas=betas, eps=eps, weight_decays=decays,
                       masters=[s["master"] for s in states])


def _check(before, after, step, decay, betas=BETAS, eps=EPS, lr=LR):
    w0 = f64(before["master"] if before["master"] is not None else before["param"])
    g, m0, v0 = f64(before["grad"]), f64(before["exp_avg"]), f64(before["exp_avg_sq"])
    d = float(np.float32(decay))
    w, m, v = O.adamw(w0, g, m0, v0, step, lr, *betas, eps, d)
    m_off = 5 * U32 * (np.abs(betas[0] * m0) + np.abs((1 - betas[0]) * g))
    v_off = 6 * U32 * v
    assert_within(after["exp_avg"], m, m_off + 1.01 * half_step(np.abs(m) + m_off, after["exp_avg"].dtype), "m")
    assert_within(after["exp_avg_sq"], v, v_off + 1.01 * half_step(v + v_off, after["exp_avg_sq"].dtype), "v")
    root = np.sqrt(v / (1 - betas[1] ** step)) + eps
    size = lr / (1 - betas[0] ** step) / np.maximum(root, 1e-300)
    off = size * (m_off + np.abs(m) * 14 * U32) + 3 * U32 * (np.abs(w0) + np.abs(w)) + 1e-12 * size
    if after["master"] is not None:
        assert_within(after["master"], w, off, "master")
        assert torch.equal(after["param"], after["master"].to(after["param"].dtype))
    else:
        assert_within(after["param"], w, off + 1.01 * half_step(np.abs(w) + off, after["param"].dtype), "w")


def _copy(s):
    return {k: (t.clone() if t is not None else None) for k, t in s.items()}


@pytest.mark.parametrize("p,g,m,v,master", [
    (SF, SF, SF, SF, False), (BF, BF, SF, SF, True), (BF, BF, BF, BF, False), (HF, HF, SF, SF, True),
    (HF, SF, HF, BF, False), (SF, BF, BF, SF, False), (SF, SF, SF, SF, True)])
def test_step(p, g, m, v, master):
    require_gpu()
    shapes = [(1,), (7,), (4096,), (4097,), (33, 129), (2, 3, 5), (8191,), (100, 1000)]
    states = [_state(10 * i, sh, p, g, m, v, master) for i, sh in enumerate(shapes)]
    decays = [0.1 * (i % 3) for i in range(len(shapes))]
    for step in (1, 2, 100000):
        before = [_copy(s) for s in states]
        _step(states, step, decays)
        for b, s, d in zip(before, states, decays):
            _check(b, s, step, d)
            assert torch.equal(b["grad"], s["grad"])


def test_many_tensors_of_mixed_types_equal_single_calls():
    """More tensors than one launch holds; each equals its own call, bitwise."""
    require_gpu()
    types = [(SF, SF, SF, SF, False), (BF, BF, SF, SF, True), (HF, SF, BF, BF, False)]
    states = [_state(i, (1 + 977 * i,), *types[i % 3]) for i in range(75)]
    alone = [_copy(s) for s in states]
    empty = _state(1, (0,), *types[0])
    _step(states[:40] + [empty] + states[40:], 3, [0.01] * 76)
    for s, a in zip(states, alone):
        _step([a], 3, [0.01])
        for k in s:
            assert s[k] is None or torch.equal(s[k], a[k]), k


def test_unaligned_tensors_and_their_surroundings():
    require_gpu()
    store = {k: torch.full((9000,), 7.0, dtype=SF if k == "v" else BF, device="cuda") for k in "pgmv"}
    part = {k: t[3:8998] for k, t in store.items()}
    for i, k in enumerate("pgmv"):
        part[k].copy_(normal(i, (8995,), SF, 0.1).abs())
    s = dict(param=part["p"], grad=part["g"], exp_avg=part["m"], exp_avg_sq=part["v"], master=None)
    before = _copy(s)
    _step([s], 4, [0.1])
    _check(before, s, 4, 0.1)
    for t in store.values():
        assert torch.all(t[:3] == 7) and torch.all(t[8998:] == 7)


def test_zero_gradients_infinities_and_options():
    require_gpu()
    s = _state(1, (5000,), SF, SF, SF, SF, False)
    for t in (s["grad"], s["exp_avg"], s["exp_avg_sq"]):
        t[:100] = 0
    s["grad"][200], s["grad"][201] = float("inf"), float("nan")
    before = _copy(s)
    _step([s], 1, [0.0])
    assert torch.equal(s["param"][:100], before["param"][:100])      # 0 / eps
    assert torch.isnan(s["param"][200:202]).all() and torch.isfinite(s["param"][:200]).all()
    for betas, eps, lr in (((0.0, 0.0), 1e-3, 0.1), ((0.5, 0.9), 0.5, 1.0), ((0.9, 0.95), 1e-8, 0.0)):
        s = _state(2, (3000,), SF, SF, SF, SF, False)
        before = _copy(s)
        _step([s], 7, [0.2], betas=betas, eps=eps, lr=lr)
        _check(before, s, 7, 0.2, betas=betas, eps=eps, lr=lr)
        if lr == 0.0:
            assert torch.equal(s["param"], before["param"])


def test_offsets_beyond_32_bits():
    require_gpu()
    n = (1 << 31) + 4099
    p = torch.zeros(n, dtype=BF, device="cuda")
    m, v, g = torch.zeros_like(p), torch.zeros_like(p), torch.zeros_like(p)
    g[-1], g[5], g[-5000] = 1.0, 1.0, -1.0
    nsmi.ns_adamw_step([p], [g], [m], [v], step=1, lr=0.5, eps=0.0, betas=(0.5, 0.5))
    # zero gradients from zero states with eps = 0 are 0 / 0
    assert [p[-1].item(), p[5].item(), p[-5000].item()] == [-0.5, -0.5, 0.5]
    assert torch.isnan(p[-2]).item() and m[-1].item() == 0.5 and m[-2].item() == 0.0
