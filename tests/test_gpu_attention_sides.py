"""GPU: attention where few workgroups share a tile's keys between two halves of their
waves, and where they do not, on both sides of the rule: 384 rows a sequence on average."""

import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_attention import check, check_grad, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[384], [385], [23], [40, 728], [0, 768], [1155, 0, 0], [1, 1, 1150], [1100, 1, 60]],
                         ids=str)
@pytest.mark.parametrize("shape", [(4, 2, 128), (3, 1, 64), (6, 2, 80)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_both_sides_of_the_rule(lengths, shape, dtype):
    require_gpu()
    c = make(sum(lengths), lengths, *shape, dtype, rest=3)
    check(c)
    check_grad(c)
    peaked = make(sum(lengths) + 1, lengths, *shape, dtype, peak=20.0)
    check(peaked)
    check_grad(peaked)
