"""How the operators around the matrix update are called: Python refusals on
GPU tensors, other streams, HIP graph replays, reproducibility.

A replay is checked against an eager call of the same inputs, several times,
with the inputs overwritten in place and eager work in between.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from train_helpers import normal

pytestmark = pytest.mark.gpu

BF, SF = torch.bfloat16, torch.float32


class Step:
    """Every operator once, on fixed buffers."""

    def __init__(self, seed, tokens=96, rows=1500, dim=200):
        pairs, length = 2, tokens // 4
        self.table = normal(seed, (rows, dim), BF)
        self.w = normal(seed + 1, (dim,), BF)
        self.res = normal(seed + 2, (tokens, dim), BF)
        g = torch.Generator().manual_seed(seed)
        self.ids = torch.randint(0, rows, (tokens,), generator=g).cuda()
        self.labels = torch.randint(-20, rows, (2 * pairs, length), generator=g).cuda()
        self.logits = normal(seed + 3, (2 * pairs, length, rows), BF)
        self.ref = normal(seed + 4, (2 * pairs,))
        self.m, self.v = torch.zeros(rows, dim, device="cuda"), torch.zeros(rows, dim, device="cuda")
        self.inputs = [self.table, self.w, self.res, self.ids, self.labels, self.logits, self.ref,
                       self.m, self.v]

    def __call__(self):
        x = nsmi.ns_embedding(self.table, self.ids, scale=3.0)
        y, h, rstd = nsmi.ns_rms_norm(x, self.w, residual=self.res)
        q, scales, _, _ = nsmi.ns_rms_norm_fp8(x, self.w, residual=self.res)
        losses, margins, logps, lse = nsmi.ns_preference_loss(self.logits, self.labels, self.ref)
        dlogits = nsmi.ns_preference_loss_grad(self.logits, self.labels, margins, lse, losses)
        dx, dw = nsmi.ns_rms_norm_grad(y, h, self.w, rstd, dh=self.res)
        dtable = nsmi.ns_embedding_grad(dx, self.ids, self.table.shape[0], scale=3.0, out_dtype=SF)
        nsmi.ns_adamw_step([self.table, self.w], [dtable, dw], [self.m, torch.zeros_like(self.w)],
                           [self.v, torch.zeros_like(self.w)], step=2, lr=1e-2)
        return [x, y, h, rstd, q.view(torch.uint8), scales, losses, margins, logps, lse, dlogits, dx,
                dw, dtable, self.table.clone(), self.w.clone(), self.m.clone(), self.v.clone()]


def _same(a, b):
    return [i for i, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y)]


def test_graph_replays_equal_eager_calls():
    require_gpu()
    step = Step(1)
    fresh = [t.clone() for t in step.inputs]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        other = Step(50 + k)
        for t, o, f in zip(step.inputs, other.inputs, fresh):
            t.copy_(o if k % 2 else f)
        if k % 2:
            want = other()
        else:
            again = Step(1)
            want = again()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, want) == [], k


def test_calls_on_two_streams():
    require_gpu()
    steps = [Step(10), Step(20, tokens=400), Step(30, rows=5000), Step(40, dim=65)]
    want = [Step(10)(), Step(20, tokens=400)(), Step(30, rows=5000)(), Step(40, dim=65)()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for k, s in enumerate(steps):
        with torch.cuda.stream(streams[k % 2]):
            got.append(s())
    torch.cuda.synchronize()
    for k in range(4):
        assert _same(got[k], want[k]) == [], k


def test_given_workspaces_need_no_contents():
    require_gpu()
    g, ids = normal(1, (3000, 48)), torch.randint(0, 90, (3000,)).cuda()
    want = nsmi.ns_embedding_grad(g, ids, 90)
    n = nsmi.ns_embedding_grad_workspace_size(90, 48, 3000)
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(nsmi.ns_embedding_grad(g, ids, 90, workspace=ws), want)
    w, h = normal(2, (48,)), normal(3, (3000, 48))
    _, _, rstd = nsmi.ns_rms_norm(h, w)
    dx, dw = nsmi.ns_rms_norm_grad(g, h, w, rstd)
    ws = torch.full((nsmi.ns_rms_norm_grad_workspace_size(3000, 48),), 255, dtype=torch.uint8,
                    device="cuda")
    dx2, dw2 = nsmi.ns_rms_norm_grad(g, h, w, rstd, workspace=ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    logits, labels = normal(4, (2, 5, 60000)), torch.randint(-9, 60000, (2, 5)).cuda()
    ref = torch.zeros(2, device="cuda")
    want = nsmi.ns_preference_loss(logits, labels, ref)
    ws = torch.full((nsmi.ns_preference_loss_workspace_size(1, 5, 60000),), 255, dtype=torch.uint8,
                    device="cuda")
    assert _same(nsmi.ns_preference_loss(logits, labels, ref, workspace=ws), want) == []


def test_refusals_on_gpu_tensors():
    require_gpu()
    x, w = normal(1, (6, 16)), normal(2, (16,))
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    rstd = torch.ones(6, device="cuda")
    logits, labels = normal(3, (2, 3, 16)), torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    ref = torch.zeros(2, device="cuda")
    bad = [
        (TypeError, lambda: nsmi.ns_embedding(x, ids.float())),
        (TypeError, lambda: nsmi.ns_embedding(x.double(), ids)),
        (ValueError, lambda: nsmi.ns_embedding(x.t(), ids)),
        (ValueError, lambda: nsmi.ns_embedding(x, ids, out=x[:, :8])),
        (ValueError, lambda: nsmi.ns_embedding(x, ids.cpu())),
        (nsmi.NsError, lambda: nsmi.ns_embedding(x, ids, out=x)),
        (nsmi.NsError, lambda: nsmi.ns_embedding(x, ids, scale=float("nan"))),
        (ValueError, lambda: nsmi.ns_embedding_grad(x, ids[:5], 9)),
        (ValueError, lambda: nsmi.ns_embedding_grad(x, ids, 9, accumulate=True)),
        (ValueError, lambda: nsmi.ns_embedding_grad(x, ids, 9, padding_idx=9)),
        (ValueError, lambda: nsmi.ns_embedding_grad(x, ids, 9, out=x)),
        (TypeError, lambda: nsmi.ns_embedding_grad(x, ids, 6, out=x.clone(), out_dtype=BF)),
        (nsmi.NsError, lambda: nsmi.ns_embedding_grad(x, ids, 0)),
        (ValueError, lambda: nsmi.ns_rms_norm(x, w[:8])),
        (ValueError, lambda: nsmi.ns_rms_norm(x, w, residual=x[:5])),
        (ValueError, lambda: nsmi.ns_rms_norm(x, w, h=x)),
        (ValueError, lambda: nsmi.ns_rms_norm(x[:, None, :].expand(6, 3, 16), w)),
        (nsmi.NsError, lambda: nsmi.ns_rms_norm(x, w, residual=x.to(BF))),
        (nsmi.NsError, lambda: nsmi.ns_rms_norm(x, w, eps=-1.0)),
        (TypeError, lambda: nsmi.ns_rms_norm(x, w, residual=x, h=x.to(BF))),
        (ValueError, lambda: nsmi.ns_rms_norm_grad(x, x[:5], w, rstd)),
        (TypeError, lambda: nsmi.ns_rms_norm_grad(x, x, w, rstd.double())),
        (TypeError, lambda: nsmi.ns_rms_norm_grad(x, x, w, rstd, dh=x.to(BF), dx_dtype=SF)),
        (nsmi.NsError, lambda: nsmi.ns_rms_norm_grad(x, x, w, rstd, dx=x)),
        (ValueError, lambda: nsmi.ns_preference_loss(logits, labels[:1], ref)),
        (ValueError, lambda: nsmi.ns_preference_loss(logits, labels, ref[:1])),
        (TypeError, lambda: nsmi.ns_preference_loss(logits, labels, ref.double())),
        (nsmi.NsError, lambda: nsmi.ns_preference_loss(logits, labels, ref, label_smoothing=2.0)),
        (ValueError, lambda: nsmi.ns_preference_loss_grad(logits, labels, ref, ref, ref)),
        (TypeError, lambda: nsmi.ns_preference_loss_grad(logits, labels, ref[:1], torch.zeros(
            (2, 3), device="cuda"), ref[:1], out=logits.to(BF))),
        (ValueError, lambda: nsmi.ns_adamw_step([x], [x.clone()], [x[:3]], [x.clone()], 1, 0.1)),
        (ValueError, lambda: nsmi.ns_adamw_step([x.t()], [x.t()], [x.t()], [x.t()], 1, 0.1)),
        (nsmi.NsError, lambda: nsmi.ns_adamw_step([x], [x], [x.clone()], [x.clone()], 1, 0.1)),
        (nsmi.NsError, lambda: nsmi.ns_adamw_step([x], [x.clone()], [x.clone()], [x.clone()], 0, 0.1)),
    ]
    before = [t.clone() for t in (x, w, logits)]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"refusal {i} did not raise")
    torch.cuda.synchronize()
    assert _same(before, [x, w, logits]) == []
