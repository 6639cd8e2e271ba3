"""How the operators on heads and the token log probabilities are called: a run of
them together, HIP graph replays, other streams, given workspaces, refusals on GPU
tensors, reproducibility.

A replay is checked against an eager call of the same inputs, several times, with
the inputs (the sequences' offsets among them) overwritten in place and eager work
in between.
"""

import pytest
import torch

import newton_schulz_matrix_amd as nsmi
from gpu_helpers import require_gpu
from train_helpers import normal

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


class Layer:
    """Every operator once, on fixed buffers, as a layer and a loss use them."""

    def __init__(self, seed, tokens=300, lengths=(100, 37, 0, 150), heads=(6, 2), dim=64, vocab=1500, dtype=BF, top=5):
        hq, hk = heads
        g = torch.Generator().manual_seed(seed)
        self.heads, self.top = (hq, hk, hk), top
        self.qkv = normal(seed, (tokens, hq + 2 * hk, dim), dtype)
        self.weights = normal(seed + 1, (2, dim), dtype)
        self.at = torch.randint(0, 5000, (3, tokens), generator=g).cuda()
        self.freq = torch.rand(dim // 2, generator=g).cuda()
        self.ends = torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32, device="cuda")
        self.logits = normal(seed + 2, (tokens, vocab), dtype, 3.0)
        self.tokens = torch.randint(-300, vocab, (tokens,), generator=g).cuda()
        self.sections = [dim // 2 - 2 * (dim // 8), dim // 8, dim // 8]
        self.inputs = [self.qkv, self.weights, self.at, self.freq, self.ends, self.logits, self.tokens]

    def __call__(self):
        q0, k0, v = self.qkv.split(self.heads, 1)
        turn = dict(sections=self.sections)
        q, k = nsmi.ns_qk_norm_rope(q0, k0, *self.weights, self.at, self.freq, **turn)
        out, lse = nsmi.ns_attention(q, k, v, self.ends)
        d = torch.empty_like(self.qkv).zero_()
        dq, dk, dv = d.split(self.heads, 1)
        nsmi.ns_attention_grad(out, q, k, v, out, lse, self.ends, dq=dq, dk=dk, dv=dv)
        raw = d.clone()
        _, _, dqw, dkw = nsmi.ns_qk_norm_rope_grad(dq, dk, q0, k0, *self.weights, self.at, self.freq, dq=dq, dk=dk, **turn)
        logps, z, entropy, best, ids = nsmi.ns_token_logps(self.logits, self.tokens, top=self.top)
        dlogits = nsmi.ns_token_logps_grad(self.logits, self.tokens, z, entropy, logps, dentropy=entropy)
        return [q, k, out, lse, raw, d, dqw, dkw, logps, z, entropy, best, ids, dlogits]


def _same(a, b):
    return [i for i, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y)]


CASES = [dict(), dict(dtype=HF, dim=128), dict(tokens=1600, lengths=(1100, 0, 317, 1), heads=(2, 1), dim=80),
         dict(tokens=40, lengths=(5, 20), vocab=30000, top=20)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_graph_replays_equal_eager_calls(case):
    require_gpu()
    layer = Layer(1, **case)
    fresh = [t.clone() for t in layer.inputs]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    shorter = dict(case, lengths=tuple(n // 2 for n in case.get("lengths", (100, 37, 0, 150))))
    for k in range(4):
        other = Layer(50 + k, **shorter) if k % 2 else Layer(1, **case)
        for t, o, f in zip(layer.inputs, other.inputs, fresh):
            t.copy_(o if k % 2 else f)
        want = other()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, want) == [], k


def test_two_graphs_with_workspaces_of_their_own():
    """Graphs captured one after the other and replayed on two streams at once."""
    require_gpu()
    layers, graphs, outs = [Layer(3), Layer(4, **CASES[2])], [], []
    want = [layer() for layer in layers]
    torch.cuda.synchronize()
    for layer in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer())
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], want[0]) == [] and _same(outs[1], want[1]) == []
        layers[0]()


def test_calls_on_two_streams():
    require_gpu()
    layers = [Layer(10 + k, **case) for k, case in enumerate(CASES)]
    want = [Layer(10 + k, **case)() for k, case in enumerate(CASES)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for k, layer in enumerate(layers):
        with torch.cuda.stream(streams[k % 2]):
            got.append(layer())
    torch.cuda.synchronize()
    for k in range(len(CASES)):
        assert _same(got[k], want[k]) == [], k


def test_given_workspaces_need_no_contents():
    require_gpu()
    for dtype, heads in ((BF, (6, 2)), (HF, (2, 1))):
        layer = Layer(20, tokens=1500, lengths=(1200, 200), heads=heads, dtype=dtype)
        q, k, v = (x.contiguous() for x in layer.qkv.split(layer.heads, 1))
        w = layer.weights

        def calls(fill):
            def ws(n):
                return None if fill is None else torch.full((max(n, 1),), fill, dtype=torch.uint8, device="cuda")
            sizes = (1500, 2, *heads, 64)
            out, lse = nsmi.ns_attention(q, k, v, layer.ends, workspace=ws(nsmi.ns_attention_workspace_size(*sizes)))
            grads = nsmi.ns_attention_grad(out, q, k, v, out, lse, layer.ends,
                                           workspace=ws(nsmi.ns_attention_grad_workspace_size(*sizes)))
            turned = nsmi.ns_qk_norm_rope_grad(q, k, q, k, *w, layer.at[0], layer.freq,
                                               workspace=ws(nsmi.ns_qk_norm_rope_grad_workspace_size(1500, 64)))
            rows = layer.logits[:4], layer.tokens[:4]
            found = nsmi.ns_token_logps(*rows, top=7, workspace=ws(nsmi.ns_token_logps_workspace_size(4, 1500, 7)))
            return [out, lse, *grads, *turned, *found]

        want = calls(None)
        for fill in (0, 255, 127):
            assert _same(calls(fill), want) == [], (dtype, fill)


def test_refusals_on_gpu_tensors():
    require_gpu()
    x, w = normal(1, (6, 4, 16), BF), normal(2, (16,), BF)
    k, at, f = normal(3, (6, 2, 16), BF), torch.arange(6, device="cuda"), torch.rand(8).cuda()
    ends = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    lse = torch.zeros((4, 6), device="cuda")
    z, ids, rows = normal(4, (6, 32), BF), torch.arange(6, device="cuda"), torch.zeros(6, device="cuda")
    norm, grad = nsmi.ns_qk_norm_rope, nsmi.ns_qk_norm_rope_grad
    attn, agrad = nsmi.ns_attention, nsmi.ns_attention_grad
    bad = [
        (TypeError, lambda: norm(x, k.float(), w, w, at, f)),
        (ValueError, lambda: norm(x, k[:5], w, w, at, f)),
        (ValueError, lambda: norm(x, k, w, None, at, f)),
        (ValueError, lambda: norm(x, k, w[:8], w[:8], at, f)),
        (TypeError, lambda: norm(x, k, w, w.float(), at, f)),
        (nsmi.NsError, lambda: norm(x, k, w.to(HF), w.to(HF), at, f)),
        (ValueError, lambda: norm(x, k, w, w, at[:5], f)),
        (TypeError, lambda: norm(x, k, w, w, at.float(), f)),
        (TypeError, lambda: norm(x, k, w, w, at, f.double())),
        (ValueError, lambda: norm(x, k, w, w, at, f[None])),
        (ValueError, lambda: norm(x, k, w, w, at.cpu(), f)),
        (nsmi.NsError, lambda: norm(x, k, w, w, at, f[:7])),
        (nsmi.NsError, lambda: norm(x, k, w, w, at, torch.rand(10).cuda())),
        (ValueError, lambda: norm(x, k, w, w, at.expand(2, 6), f)),
        (ValueError, lambda: norm(x, k, w, w, at.expand(2, 6), f, sections=[4, 3])),
        (ValueError, lambda: norm(x, k, w, w, at.expand(5, 6), f, sections=[4, 1, 1, 1, 1])),
        (ValueError, lambda: norm(x, k, w, w, at, f, sections=[4, 4])),
        (nsmi.NsError, lambda: norm(x, k, w, w, at, f, eps=-1.0)),
        (ValueError, lambda: norm(x.transpose(1, 2), k, w, w, at, f)),
        (ValueError, lambda: norm(x, k, w, w, at, f, out_q=x[:5])),
        (TypeError, lambda: norm(x, k, w, w, at, f, out_q=x.float())),
        (nsmi.NsError, lambda: norm(x, k, w, w, at, f, out_q=x[:, :1].expand(6, 4, 16))),
        (nsmi.NsError, lambda: norm(x, x[:, :2], w, w, at, f, out_q=x)),
        (ValueError, lambda: grad(x[:5], k, x, k, w, w, at, f)),
        (TypeError, lambda: grad(x.float(), k, x, k, w, w, at, f)),
        (nsmi.NsError, lambda: grad(x, k, x, k, w, w, at, f, dq=x)),      # over the call's input
        (ValueError, lambda: attn(x, k, k[:5], ends)),
        (ValueError, lambda: attn(x, k[:, :, :8], k[:, :, :8], ends)),
        (TypeError, lambda: attn(x, k, k.to(HF), ends)),
        (nsmi.NsError, lambda: attn(x.float(), k.float(), k.float(), ends)),
        (nsmi.NsError, lambda: attn(x[:, :3], k, k, ends)),
        (TypeError, lambda: attn(x, k, k, ends.long())),
        (ValueError, lambda: attn(x, k, k, ends[:0])),
        (ValueError, lambda: attn(x, k, k, ends.cpu())),
        (nsmi.NsError, lambda: attn(x, k, k, ends, scale=-1.0)),
        (nsmi.NsError, lambda: attn(x, k, k, ends, out=x)),
        (nsmi.NsError, lambda: attn(x[:, :, :12], k[:, :, :12], k[:, :, :12], ends)),
        (nsmi.NsError, lambda: attn(x[1:, :, 4:12], k[1:, :, :8], k[1:, :, :8], ends)),   # 8-byte aligned
        (ValueError, lambda: agrad(x, x, k, k, x, lse[:3], ends)),
        (TypeError, lambda: agrad(x, x, k, k, x, lse.double(), ends)),
        (ValueError, lambda: agrad(x, x, k, k, x, lse, ends, dq=x.clone())),
        (nsmi.NsError, lambda: agrad(x, x, k, k, x, lse, ends, dq=x.clone(), dk=k, dv=k.clone())),
        (TypeError, lambda: nsmi.ns_token_logps(z, ids.float())),
        (ValueError, lambda: nsmi.ns_token_logps(z, ids[:5])),
        (nsmi.NsError, lambda: nsmi.ns_token_logps(z, ids, top=33)),
        (nsmi.NsError, lambda: nsmi.ns_token_logps(normal(5, (2, 99), BF), ids[:2], top=65)),
        (ValueError, lambda: nsmi.ns_token_logps(z.t(), ids)),
        (ValueError, lambda: nsmi.ns_token_logps_grad(z, ids, rows, None, rows, dentropy=rows)),
        (TypeError, lambda: nsmi.ns_token_logps_grad(z, ids, rows, rows, rows, out=z.float())),
        (ValueError, lambda: nsmi.ns_token_logps_grad(z, ids, rows[:3], rows, rows)),
    ]
    before = [t.clone() for t in (x, k, z)]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"refusal {i} did not raise")
    torch.cuda.synchronize()
    assert _same(before, [x, k, z]) == []
