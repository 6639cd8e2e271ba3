"""A preference-training step in which every parameter is this library's.

A small model (embedding, norm, two matrices, norm with the residual, head)
learns to prefer one of two continuations. Its two matrices take the Muon
step; the embedding table, the head and the norm gains take AdamW. The
products of the layers are torch's; the backward pass is written out, call by
call. Run it on an MI355X:

    python examples/preference_training.py
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import newton_schulz_matrix_amd as nsmi  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class Model:
    """Weights in bf16 with fp32 copies where AdamW updates them."""

    def __init__(self, vocab=1000, dim=256, hidden=768, seed=0):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
        self.scale = dim ** 0.5
        self.masters = {"table": normal(vocab, dim) / dim ** 0.5, "head": normal(vocab, dim) / dim ** 0.5,
                        "gain1": torch.ones(dim, device="cuda"), "gain2": torch.ones(dim, device="cuda")}
        self.w = {k: t.to(BF) for k, t in self.masters.items()}
        self.moments = {k: (torch.zeros_like(t), torch.zeros_like(t)) for k, t in self.masters.items()}
        self.mats = {"up": (normal(hidden, dim) / dim ** 0.5).to(BF),
                     "down": (normal(dim, hidden) / hidden ** 0.5).to(BF)}
        self.momenta = {k: torch.zeros_like(t) for k, t in self.mats.items()}
        self.steps = 0

    def forward(self, ids):
        """Logits of ids (sequences, length) and what the backward pass needs."""
        w, m, s = self.w, self.mats, {"ids": ids}
        x = nsmi.ns_embedding(w["table"], ids.reshape(-1), scale=self.scale)
        s["y1"], s["h1"], s["r1"] = nsmi.ns_rms_norm(x, w["gain1"])
        s["a"] = s["y1"] @ m["up"].t()
        s["b"] = s["a"].relu()
        c = s["b"] @ m["down"].t()
        s["y2"], s["h2"], s["r2"] = nsmi.ns_rms_norm(c, w["gain2"], residual=s["h1"])
        return (s["y2"] @ w["head"].t()).view(*ids.shape, -1), s

    def backward(self, s, dlogits):
        """Gradients of every parameter."""
        w, m, g = self.w, self.mats, {}
        dlogits = dlogits.flatten(0, 1)
        g["head"] = dlogits.t() @ s["y2"]
        dc, g["gain2"] = nsmi.ns_rms_norm_grad(dlogits @ w["head"], s["h2"], w["gain2"], s["r2"],
                                               dweight_dtype=F32)
        g["down"] = dc.t() @ s["b"]
        da = (dc @ m["down"]) * (s["a"] > 0)
        g["up"] = da.t() @ s["y1"]
        dx, g["gain1"] = nsmi.ns_rms_norm_grad(da @ m["up"], s["h1"], w["gain1"], s["r1"], dh=dc,
                                               dweight_dtype=F32)
        g["table"] = nsmi.ns_embedding_grad(dx, s["ids"].reshape(-1), w["table"].shape[0],
                                            scale=self.scale)
        return g

    def update(self, g, lr=1e-3, muon_lr=2e-2):
        self.steps += 1
        mats = list(self.mats)
        nsmi.ns_muon_step([g[k] for k in mats], [self.momenta[k] for k in mats],
                          [self.mats[k] for k in mats], beta=0.9, lr=muon_lr, scales=[0.2] * len(mats))
        rest = list(self.w)
        nsmi.ns_adamw_step([self.w[k] for k in rest], [g[k] for k in rest],
                           [self.moments[k][0] for k in rest], [self.moments[k][1] for k in rest],
                           step=self.steps, lr=lr, betas=(0.9, 0.95),
                           weight_decays=[0.01 if self.w[k].dim() == 2 else 0.0 for k in rest],
                           masters=[self.masters[k] for k in rest])


def batch(pairs=8, length=64, vocab=1000, seed=1):
    """Ids (2 pairs, length) and the labels of the continuations: both of a
    pair share a prompt; its positions do not count."""
    g = torch.Generator().manual_seed(seed)
    prompt = torch.randint(0, vocab, (pairs, length // 2), generator=g).repeat(2, 1)
    ids = torch.cat([prompt, torch.randint(0, vocab, (2 * pairs, length - length // 2), generator=g)], 1)
    labels = torch.roll(ids, -1, 1)
    labels[:, :length // 2 - 1] = -100
    labels[:, -1] = -100
    return ids.cuda(), labels.cuda()


def train(steps=20, beta=0.1):
    model = Model()
    ids, labels = batch()
    pairs = ids.shape[0] // 2
    zero = torch.zeros(2 * pairs, device="cuda")
    # the reference is the model as it starts
    reference = nsmi.ns_preference_loss(model.forward(ids)[0], labels, zero)[2].clone()
    weights = torch.full((pairs,), 1.0 / pairs, device="cuda")
    history = []
    for _ in range(steps):
        logits, saved = model.forward(ids)
        losses, margins, _, lse = nsmi.ns_preference_loss(logits, labels, reference, beta=beta)
        dlogits = nsmi.ns_preference_loss_grad(logits, labels, margins, lse, weights, beta=beta,
                                               out=logits)
        model.update(model.backward(saved, dlogits))
        history.append(losses.mean().item())
    return history


if __name__ == "__main__":
    for i, loss in enumerate(train()):
        print(f"step {i:2d}  loss {loss:.4f}")
