"""Lookups of so many ids that a workgroup takes four rows a team, by several
teams: a lookup is one product and one rounding."""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from train_helpers import normal, strided_rows, untouched

pytestmark = pytest.mark.gpu

BF, SF = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dim,count", [(1001, 8197), (512, 16390), (100, 65550), (24, 262151), (5, 1048583)])
@pytest.mark.parametrize("dtype", [BF, SF])
def test_lookup_of_many_ids(dim, count, dtype):
    require_gpu()
    print("lookup of many ids", dim, count, dtype, flush=True)
    rows = 333
    table = normal(dim, (rows, dim), dtype)
    g = torch.Generator().manual_seed(count)
    ids = torch.randint(-30, rows + 30, (count,), generator=g).cuda()
    inside = (ids >= 0) & (ids < rows)
    want = table[ids.clamp(0, rows - 1)].float() * 1.5 * inside[:, None]
    assert torch.equal(nsmi.ns_embedding(table, ids, scale=1.5), want.to(dtype))
    if dim > 100:
        out, store = strided_rows(torch.zeros(count, dim, dtype=dtype, device="cuda"), 3, 5)
        nsmi.ns_embedding(table, ids.to(torch.int32), scale=1.5, out=out)
        assert torch.equal(out, want.to(dtype)) and untouched(store, out)
