"""The preference-training example: its hand-written backward pass against
fp64 autograd of the same model, and a falling loss."""

import os
import sys

import pytest
import torch

from gpu_helpers import require_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gradients_of_the_whole_step():
    """bf16 activations round about ten times on the way: 2^-8 each, so the
    gradients' relative errors stay below a tenth."""
    require_gpu()
    import newton_schulz_matrix_amd as nsmi
    import preference_training as E
    model, (ids, labels) = E.Model(), E.batch()
    pairs = ids.shape[0] // 2
    ref = torch.linspace(-3, 3, 2 * pairs).cuda() - 32 * 6.9
    weights = torch.full((pairs,), 1.0 / pairs, device="cuda")
    logits, saved = model.forward(ids)
    losses, margins, _, lse = nsmi.ns_preference_loss(logits, labels, ref)
    got = model.backward(saved, nsmi.ns_preference_loss_grad(logits, labels, margins, lse, weights))
    leaves = {k: t.double().cpu().requires_grad_() for k, t in {**model.w, **model.mats}.items()}

    def norm(x, w):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w

    x = leaves["table"][ids.cpu()] * model.scale
    c = (norm(x, leaves["gain1"]) @ leaves["up"].t()).relu() @ leaves["down"].t()
    logp = (norm(c + x, leaves["gain2"]) @ leaves["head"].t()).log_softmax(-1)
    lab = labels.cpu()
    token = logp.gather(-1, lab.clamp(min=0)[..., None])[..., 0]
    seq = torch.where(lab >= 0, token, torch.zeros_like(token)).sum(-1) - ref.double().cpu()
    want = -torch.nn.functional.logsigmoid(0.1 * (seq[:pairs] - seq[pairs:]))
    want.mean().backward()
    assert torch.allclose(losses.double().cpu(), want.detach(), rtol=0.1, atol=0.05)
    for k, t in leaves.items():
        err = (got[k].double().cpu() - t.grad).norm() / t.grad.norm()
        assert err < 0.1, (k, err.item())


def test_the_loss_falls():
    require_gpu()
    import preference_training as E
    history = E.train(steps=15)
    assert history[0] == pytest.approx(0.6931, abs=1e-3) and history[-1] < 0.5 * history[0]
