"""Embedding lookup and its gradient against the fp64 forms.

Tolerances. The lookup rounds the fp32 product and then the output once: half
a step of each. A gradient element is a fixed-order fp32 sum of n terms: at
most n + 2 roundings (the sum, the scale, the addition to the old value), each
half a step of a partial sum no larger than the sum of magnitudes, then one
rounding to the output type.
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


def _ids(seed, count, rows, skew=True):
    rng = np.random.default_rng(seed)
    if skew:
        ids = np.floor(np.exp(rng.random(count) * np.log(rows + 1))) - 1
    else:
        ids = rng.integers(0, rows, count)
    return np.clip(ids, 0, rows - 1).astype(np.int64)


@pytest.mark.parametrize("rows,dim,count,dtype,out,scale", [
    (1, 1, 1, SF, SF, 1.0), (5, 7, 3, BF, BF, 0.3), (300, 64, 1, HF, SF, 2.0),
    (1000, 513, 77, BF, BF, 1.0), (97, 2049, 40, SF, HF, 0.7), (50021, 1001, 4099, HF, BF, 11.3),
    (64, 4096, 9000, BF, BF, 64.0), (33, 24, 70000, SF, SF, 1.0), (12, 65536, 5, BF, SF, 1.0),
])
@pytest.mark.parametrize("int32", [False, True])
def test_lookup(rows, dim, count, dtype, out, scale, int32):
    require_gpu()
    print("lookup", rows, dim, count, dtype, out, flush=True)
    table = normal(rows + dim, (rows, dim), dtype)
    ids = _ids(count, count, rows, skew=False)
    ids[::5] = np.where(np.arange(count) % 2 == 0, -1, rows)[::5]      # outside the table
    got = nsmi.ns_embedding(table, torch.from_numpy(ids).to(torch.int32 if int32 else torch.int64)
                            .cuda(), scale=scale, out_dtype=out)
    want = O.embedding(f64(table), ids, float(np.float32(scale)))
    assert got.dtype == out
    assert_within(got, want, U32 * np.abs(want) * 1.01 + 1.01 * half_step(want, out))


def test_lookup_copies_exactly_and_keeps_the_ids_shape():
    require_gpu()
    table = normal(1, (40, 72), BF)
    table[3, 5], table[4, 0] = float("inf"), float("nan")
    ids = torch.tensor([[3, 4, 0], [39, 3, 3]], device="cuda")
    got = nsmi.ns_embedding(table, ids)
    assert got.shape == (2, 3, 72)
    assert torch.equal(got.view(torch.int16), table[ids].view(torch.int16))
    # a strided (non-contiguous) id tensor
    assert torch.equal(nsmi.ns_embedding(table, ids.t())[:, :, 7:].float().nan_to_num(),
                       table[ids.t()][:, :, 7:].float().nan_to_num())


def test_lookup_strided_and_unaligned():
    require_gpu()
    for dtype in (BF, SF):
        table, _ = strided_rows(normal(2, (31, 45), dtype), 6, 3)
        out, store = strided_rows(torch.zeros(20, 45, dtype=dtype, device="cuda"), 3, 5)
        ids = torch.from_numpy(_ids(3, 20, 31)).cuda()
        nsmi.ns_embedding(table, ids, out=out)
        assert torch.equal(out, table[ids])
        assert untouched(store, out)


def test_lookup_of_nothing():
    require_gpu()
    table = normal(1, (4, 8))
    assert nsmi.ns_embedding(table, torch.empty((0,), dtype=torch.int64, device="cuda")).shape == (0, 8)
    assert nsmi.ns_embedding(table, torch.empty((3, 0), dtype=torch.int32, device="cuda")).shape == (3, 0, 8)


def _check_grad(g, ids, rows, scale, got, old=None, padding=None, out=None, what=""):
    s = float(np.float32(scale))
    want, mag, n = O.embedding_grad(f64(g), ids, rows, s, padding)
    if old is not None:
        want, mag = want + old, mag + np.abs(old)
    slack = (n[:, None] + 2) * U32 * mag * 1.01
    if old is not None:
        slack = np.where(n[:, None] == 0, 0.0, slack)
    assert_within(got, want, np.where(n[:, None] == 0, 0.0, slack + 1.01 * half_step(np.abs(want) + slack, out)),
                  what)


CASES = [
    # rows, dim, count, in, out, scale, skewed
    (1, 1, 1, SF, SF, 1.0, True), (1, 9, 500, BF, BF, 0.5, True), (2, 33, 64, HF, SF, 1.0, True),
    (255, 40, 1000, BF, SF, 2.0, False), (256, 17, 63, SF, SF, 1.0, True),
    (257, 100, 65, SF, HF, 1.0, False), (1000, 513, 4099, HF, SF, 0.3, True),
    (50021, 129, 4099, BF, BF, 1.0, True), (131072, 8, 3000, SF, SF, 1.0, True),
    (131073, 16, 3000, SF, BF, 1.0, False), (700000, 8, 300, BF, SF, 1.0, True),
    (3, 2049, 700, SF, SF, 1.0, True), (5000, 64, 70001, SF, SF, 1.0, True),
]


@pytest.mark.parametrize("rows,dim,count,dtype,out,scale,skew", CASES)
def test_gradient(rows, dim, count, dtype, out, scale, skew):
    require_gpu()
    print("gradient", rows, dim, count, dtype, out, flush=True)
    g = normal(rows + count, (count, dim), dtype)
    ids = _ids(dim, count, rows, skew)
    dev = torch.from_numpy(ids).cuda()
    got = nsmi.ns_embedding_grad(g, dev, rows, scale=scale, out_dtype=out)
    _check_grad(g, ids, rows, scale, got, out=out)
    again = nsmi.ns_embedding_grad(g, dev.to(torch.int32), rows, scale=scale, out_dtype=out)
    assert torch.equal(got, again), "int32 ids, or a second call, give other bits"
    # added to what is there
    old = normal(7, (rows, dim), out)
    into = old.clone()
    assert nsmi.ns_embedding_grad(g, dev, rows, scale=scale, out=into, accumulate=True) is into
    _check_grad(g, ids, rows, scale, into, old=f64(old), out=out, what="accumulated")


@pytest.mark.parametrize("spread", ["one id", "one group", "all distinct", "two ids in turn"])
def test_gradient_of_lopsided_ids(spread):
    require_gpu()
    rows, dim, count = 6000, 24, 6000
    i = np.arange(count)
    ids = {"one id": i * 0 + 4321, "one group": (i * 7 % 23) * 256 + 5, "all distinct": i[::-1].copy(),
           "two ids in turn": np.where(i % 2, 5, 5 + 256)}[spread]
    g = normal(3, (count, dim))
    got = nsmi.ns_embedding_grad(g, torch.from_numpy(ids).cuda(), rows)
    _check_grad(g, ids, rows, 1.0, got, out=SF)


def test_gradient_skips_padding_and_outside_ids():
    require_gpu()
    rows, dim, count = 300, 40, 2000
    ids = _ids(1, count, rows)
    ids[::7], ids[3::7] = -100, rows + 5
    ids[5::11] = 2 ** 40                    # beyond 32 bits
    g = normal(4, (count, dim), BF)
    g[torch.from_numpy((ids < 0) | (ids >= rows) | (ids == 0))] = float("nan")   # must not be read into a sum
    got = nsmi.ns_embedding_grad(g, torch.from_numpy(ids).cuda(), rows, padding_idx=0, out_dtype=SF)
    _check_grad(torch.nan_to_num(g, nan=0.0), ids, rows, 1.0, got, padding=0, out=SF)
    assert torch.all(got[0] == 0)
    none = torch.full((64,), -1, dtype=torch.int64, device="cuda")
    assert torch.all(nsmi.ns_embedding_grad(g[:64], none, rows) == 0)


def test_gradient_of_no_tokens():
    require_gpu()
    g, ids = torch.empty((0, 24), device="cuda"), torch.empty((0,), dtype=torch.int64, device="cuda")
    out = torch.full((50, 24), 7.0, device="cuda")
    nsmi.ns_embedding_grad(g, ids, 50, out=out, accumulate=True)
    assert torch.all(out == 7)
    nsmi.ns_embedding_grad(g, ids, 50, out=out)
    assert torch.all(out == 0)


def test_gradient_strided_and_unaligned():
    require_gpu()
    g, _ = strided_rows(normal(5, (500, 45), BF), 4, 1)
    out, store = strided_rows(torch.zeros(60, 45, dtype=BF, device="cuda"), 5, 3)
    ids = _ids(6, 500, 60)
    nsmi.ns_embedding_grad(g, torch.from_numpy(ids).cuda(), 60, out=out)
    _check_grad(g, ids, 60, 1.0, out, out=BF)
    assert untouched(store, out)


def test_gradient_is_the_transpose_of_the_lookup():
    """<grad, t> == <g, lookup(t)>: the difference of a linear map along t."""
    require_gpu()
    rows, dim, count = 400, 96, 3001
    ids = torch.from_numpy(_ids(8, count, rows)).cuda()
    g, t = normal(9, (count, dim)), normal(10, (rows, dim))
    grad = nsmi.ns_embedding_grad(g, ids, rows, scale=3.0)
    out = nsmi.ns_embedding(t, ids, scale=3.0)
    a, b = float((grad.double() * t.double()).sum()), float((g.double() * out.double()).sum())
    mag = float((g.double() * out.double()).abs().sum())
    assert abs(a - b) <= (count + 4) * U32 * mag


def test_offsets_beyond_32_bits():
    """A table and a gradient of more than 2^32 bytes (and 2^31 elements)."""
    require_gpu()
    rows, dim = 70000, 32768
    table = torch.zeros((rows, dim), dtype=BF, device="cuda")
    table[-1], table[40000] = 3.0, 2.0
    ids = torch.tensor([rows - 1, 40000, 0], device="cuda")
    assert nsmi.ns_embedding(table, ids).float().mean(1).tolist() == [3.0, 2.0, 0.0]
    g = torch.ones((3, dim), dtype=BF, device="cuda")
    nsmi.ns_embedding_grad(g, ids, rows, out=table)
    assert table[-1].float().mean().item() == 1.0 and table[40000].float().mean().item() == 1.0
    assert table[1:40000].abs().max().item() == 0 and table[40001:-1].abs().max().item() == 0
