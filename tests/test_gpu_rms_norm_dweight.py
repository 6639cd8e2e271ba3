"""The gain's gradient: the workgroups' shares are added in 64 bits.

With rstd and h of 1 every term is dy itself. Rows of more than 1024 columns
are a workgroup each here, so every share is one term and the sum is exact: in
fp32 the ones between two large terms would be lost.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 40, 257])
@pytest.mark.parametrize("dim", [1100, 4096, 8193])
def test_shares_that_cancel(rows, dim):
    require_gpu()
    h, w, rstd = torch.ones(rows, dim, device="cuda"), torch.ones(dim, device="cuda"), torch.ones(rows, device="cuda")
    dy = torch.ones(rows, dim, device="cuda")
    dy[0], dy[-1] = 2.0 ** 25, -(2.0 ** 25)
    _, dw = nsmi.ns_rms_norm_grad(dy, h, w, rstd)
    assert torch.all(dw == rows - 2)
