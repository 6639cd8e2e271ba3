"""The second moment over many AdamW steps, in fp32 and in bf16.

A bf16 value is off by at most 2^-8 of itself after a rounding, so under zero
gradients each step multiplies v by a factor between beta2 (1 - 2^-8) and
beta2 (1 + 2^-8). A rounding gives the old value back where the step's change,
(1 - beta2) |g^2 - v|, is below half a step, at most 2^-8 v: v settles within
2^-8 / (1 - beta2) of g^2, relative to itself (and 1% for the fp32 arithmetic).
In fp32 the same holds with 2^-24, three times a step.
"""

import warnings

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

BF, SF = torch.bfloat16, torch.float32


def _run(v, g, beta2, steps):
    w, m = torch.zeros_like(g), torch.zeros_like(g)
    for i in range(steps):
        nsmi.ns_adamw_step([w], [g], [m], [v], step=i + 1, lr=0.0, betas=(0.9, beta2))
    return v.double().cpu()


def _start(dtype):
    g = torch.Generator().manual_seed(3)
    return (torch.rand(5000, generator=g) * 4 + 1e-3).to(dtype).cuda()


@pytest.mark.parametrize("dtype,u", [(BF, 2.0 ** -8), (SF, 2.0 ** -22)])
@pytest.mark.parametrize("beta2", [0.9, 0.95, 0.99])
def test_second_moment_falls_and_settles(dtype, u, beta2):
    require_gpu()
    v0 = _start(dtype).double().cpu()
    steps = 200
    v = _run(_start(dtype), torch.zeros(5000, device="cuda"), beta2, steps)
    assert torch.all(v <= v0 * (beta2 * (1 + 1.01 * u)) ** steps)
    assert torch.all(v >= v0 * (beta2 * (1 - 1.01 * u)) ** steps)
    g = torch.linspace(0.5, 2.0, 5000).cuda()
    v = _run(_start(dtype), g, beta2, int(12 / (1 - beta2)))
    # what the steps themselves leave of the start: at most 4 beta2^steps
    left = 4.1 * beta2 ** int(12 / (1 - beta2))
    assert torch.all((g.double().cpu() ** 2 - v).abs() <= v * 1.01 * u / (1 - beta2) + left)


def test_fp32_second_moment_follows_a_slow_average():
    require_gpu()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        v = _run(_start(SF), torch.zeros(5000, device="cuda"), 0.999, 300)
    v0 = _start(SF).double().cpu()
    assert torch.all((v / v0 / 0.999 ** 300 - 1).abs() <= 300 * 4 * 2.0 ** -24)


def test_bf16_second_moment_of_a_slow_average_warns():
    """Nearest rounding gives it back unchanged: the caller is told."""
    require_gpu()
    with pytest.warns(RuntimeWarning, match="bf16"):
        v = _run(_start(BF), torch.zeros(5000, device="cuda"), 0.999, 3)
    assert v.shape == (5000,)
