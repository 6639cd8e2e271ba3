"""The preference-training example with an attention layer: its hand-written
backward pass against fp64 autograd of the same model."""

import os
import sys

import pytest
import torch

from gpu_helpers import require_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gradients_of_the_whole_step():
    """bf16 activations round about twenty times on the way there and back, half a
    step, 2^-8, each: if none cancels another the gradients' relative errors stay
    below 20 * 2^-8, 0.08, and what a rounding does to the values behind it at most
    doubles that."""
    require_gpu()
    import newton_schulz_matrix_amd as nsmi
    import preference_training as E
    model, (ids, labels) = E.AttentionModel(), E.batch(pairs=4, length=40)
    pairs = ids.shape[0] // 2
    ref = torch.linspace(-3, 3, 2 * pairs).cuda() - 20 * 6.9
    weights = torch.full((pairs,), 1.0 / pairs, device="cuda")
    logits, saved = model.forward(ids)
    losses, margins, _, lse = nsmi.ns_preference_loss(logits, labels, ref)
    got = model.backward(saved, nsmi.ns_preference_loss_grad(logits, labels, margins, lse, weights))
    leaves = {k: t.double().cpu().requires_grad_() for k, t in {**model.w, **model.mats}.items()}
    assert set(got) == set(leaves)

    def norm(x, w):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w

    n, length = ids.shape
    angle = torch.arange(length).double()[:, None] * model.inv_freq.double().cpu()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turned(x):
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    x = leaves["table"][ids.cpu()] * model.scale
    qkv = (norm(x, leaves["gain0"]) @ leaves["qkv"].t()).view(n, length, -1, model.head_dim)
    q, k, v = qkv.split((model.heads, model.kv_heads, model.kv_heads), 2)
    q, k = turned(norm(q, leaves["q_gain"])), turned(norm(k, leaves["k_gain"]))
    group = model.heads // model.kv_heads
    scores = torch.einsum("nqhd,nkhd->nhqk", q, k.repeat_interleave(group, 2)) * model.head_dim ** -0.5
    scores = scores.masked_fill(torch.ones(length, length, dtype=torch.bool).triu(1), float("-inf"))
    o = torch.einsum("nhqk,nkhd->nqhd", scores.softmax(-1), v.repeat_interleave(group, 2)).flatten(2)
    h1 = o @ leaves["out"].t() + x
    h2 = (norm(h1, leaves["gain1"]) @ leaves["up"].t()).relu() @ leaves["down"].t() + h1
    logp = (norm(h2, leaves["gain2"]) @ leaves["head"].t()).log_softmax(-1)
    lab = labels.cpu()
    token = logp.gather(-1, lab.clamp(min=0)[..., None])[..., 0]
    seq = torch.where(lab >= 0, token, torch.zeros_like(token)).sum(-1) - ref.double().cpu()
    want = -torch.nn.functional.logsigmoid(0.1 * (seq[:pairs] - seq[pairs:]))
    want.mean().backward()
    assert torch.allclose(losses.double().cpu(), want.detach(), rtol=0.16, atol=0.05)
    for name, t in leaves.items():
        err = (got[name].double().cpu() - t.grad).norm() / t.grad.norm()
        assert err < 0.16, (name, err.item())
    logps = nsmi.ns_token_logps(logits, labels, top=3)
    assert torch.allclose(logps[0].sum(-1).double().cpu(), (seq + ref.double().cpu()).detach(), rtol=0.02)


def test_it_runs():
    require_gpu()
    import preference_training as E
    history = E.train(steps=3, model=E.AttentionModel())
    assert history[0] == pytest.approx(0.6931, abs=1e-3) and all(h == h for h in history)
