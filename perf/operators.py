"""Measured cases of the operators around the matrix update of a training step:
the scaled token embedding and its gradient, the RMS norm with the residual's
addition (16/32-bit or e4m3 output) and its gradient, the preference loss on
logits and its gradient, and the AdamW step of the parameters that are not
matrices of the Newton-Schulz update (embedding tables, norm gains).

``own`` selects the library's kernels; otherwise ``run`` computes the same
outputs with elementary torch operations in 32 bits (64 for the sums over a
sequence), rounded once at the end.

Real use of the cases. Tokens are drawn with probability ~ 1 / (rank + 1), as
words are in text, so that a few tokens make up a large share of a batch.
Labels of the loss are -100 over each sequence's prompt and after its end.
Reference log probabilities are the policy's own plus noise, as early in a
preference run. Optimizer states are those of a step in mid-run.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3_MAX = 448.0
IGNORED = -100


def listed():
    return [
        # one new token for each of 8 served sequences: latency
        dict(name="embedding, 8 tokens", op="embedding", tokens=8, rows=32000, dim=4096,
             dtype="bf16", scale=1.0),
        # a training batch of 8 x 2048 tokens, scaled as models that tie the table with the head do
        dict(name="embedding, 16384 tokens", op="embedding", tokens=16384, rows=128000, dim=4096,
             dtype="bf16", scale=64.0),
        # its gradient: every row of the table's gradient is written, most of them zero
        dict(name="embedding gradient, 16384 tokens", op="embedding_grad", tokens=16384, rows=128000,
             dim=4096, dtype="bf16", out="bf16", scale=64.0, accumulate=False),
        # a small odd-sized model, gradients of micro-batches summed in fp32
        dict(name="embedding gradient, odd, summed", op="embedding_grad", tokens=4099, rows=50021,
             dim=1001, dtype="fp16", out="fp32", scale=1.0, accumulate=True),
        # one token for each of 4 served sequences: latency
        dict(name="rms norm, 4 rows", op="rms_norm", rows=4, dim=4096, dtype="bf16", residual=True,
             out="bf16"),
        # a training or prefill batch in front of an 8-bit product
        dict(name="rms norm to e4m3, 16384 rows", op="rms_norm", rows=16384, dim=4096, dtype="bf16",
             residual=True, out="e4m3"),
        # its backward pass, with the gradient that arrives along the residual
        dict(name="rms norm gradient, 16384 rows", op="rms_norm_grad", rows=16384, dim=4096,
             dtype="bf16", residual=True),
        # an odd width in full precision, no residual
        dict(name="rms norm gradient, odd, fp32", op="rms_norm_grad", rows=1031, dim=1111,
             dtype="fp32", residual=False),
        # evaluation of one short pair: few rows over a long vocabulary
        dict(name="preference loss, 1 short pair", op="preference", pairs=1, length=24, vocab=50021,
             dtype="bf16", smoothing=0.0),
        # a training step's loss and the gradient of its logits
        dict(name="preference loss and gradient, 2 pairs", op="preference_grad", pairs=2, length=1024,
             vocab=128000, dtype="bf16", smoothing=0.1),
        # the norm gains of a few layers: one launch of small tensors
        dict(name="adamw, 12 gains", op="adamw", rows=0, gains=12, dim=4096, dtype="fp32",
             grad="fp32", state="fp32", master=False),
        # an embedding table and some gains, 16-bit weights with fp32 copies
        dict(name="adamw, table of 64000 x 4096", op="adamw", rows=64000, gains=4, dim=4096,
             dtype="bf16", grad="bf16", state="fp32", master=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "rms_norm", "rms_norm_grad", "preference",
                     "preference_grad", "adamw"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("embedding", "embedding_grad"):
        dim = _log_uniform(rng, 33, 8192)
        rows = _log_uniform(rng, 256, min(131072, (1 << 29) // dim))
        case = dict(op=op, tokens=_log_uniform(rng, 1, min(65536, (1 << 27) // dim)), rows=rows,
                    dim=dim, dtype=dtype, scale=rng.choice([1.0, 0.5, round(math.sqrt(dim), 3)]))
        if op == "embedding_grad":
            case.update(out=rng.choice([dtype, "fp32"]), accumulate=rng.random() < 0.4)
        return case
    if op in ("rms_norm", "rms_norm_grad"):
        dim = _log_uniform(rng, 48, 16384)
        case = dict(op=op, rows=_log_uniform(rng, 1, min(65536, (1 << 27) // dim)), dim=dim,
                    dtype=dtype, residual=rng.random() < 0.6)
        if op == "rms_norm":
            case["out"] = rng.choice([dtype, "e4m3"])
        return case
    if op in ("preference", "preference_grad"):
        vocab = _log_uniform(rng, 1000, 131072)
        pairs = rng.randint(1, 8)
        length = _log_uniform(rng, 2, max(2, min(4096, (1 << 27) // vocab // pairs)))
        return dict(op=op, pairs=pairs, length=length, vocab=vocab, dtype=dtype,
                    smoothing=rng.choice([0.0, 0.1]))
    dim = _log_uniform(rng, 33, 8192)
    master = dtype != "fp32" and rng.random() < 0.5
    return dict(op=op, rows=_log_uniform(rng, 1, (1 << 26) // dim), gains=rng.randint(0, 10), dim=dim,
                dtype=dtype, grad=rng.choice([dtype, "fp32"]), state=rng.choice(["fp32", "bf16"]),
                master=master)


# ------------------------------------------------------------------- inputs

def _tokens(gen, count, rows):
    """Ids with probability ~ 1 / (rank + 1)."""
    u = torch.rand(count, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(rows + 1)) - 1).floor().long().clamp_(0, rows - 1)


def _labels(gen, case):
    """(2 pairs, length) labels: a prompt and the space after the end are ignored."""
    n, t = 2 * case["pairs"], case["length"]
    start = (torch.rand(n, 1, generator=gen, device="cuda") * 0.3 * t).long()
    end = t - (torch.rand(n, 1, generator=gen, device="cuda") * 0.4 * t).long()
    at = torch.arange(t, device="cuda")[None]
    labels = torch.randint(0, case["vocab"], (n, t), generator=gen, device="cuda")
    return torch.where((at >= start) & (at < end), labels, torch.full_like(labels, IGNORED))


def _adamw_shapes(case):
    shapes = [(case["rows"], case["dim"])] if case["rows"] else []
    return shapes + [(case["dim"],)] * case["gains"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, scale=1.0, mean=0.0):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(mean).to(DT[dtype])

    op, s = case["op"], {"case": case}
    if op == "embedding":
        s["table"] = normal((case["rows"], case["dim"]), case["dtype"], 0.02)
        s["ids"] = _tokens(gen, case["tokens"], case["rows"])
    elif op == "embedding_grad":
        s["grad"] = normal((case["tokens"], case["dim"]), case["dtype"], 0.01)
        s["ids"] = _tokens(gen, case["tokens"], case["rows"])
        s["into"] = (normal((case["rows"], case["dim"]), case["out"], 0.01)
                     if case["accumulate"] else None)
    elif op in ("rms_norm", "rms_norm_grad"):
        shape = (case["rows"], case["dim"])
        s["weight"] = normal((case["dim"],), case["dtype"], 0.1, 1.0)
        if op == "rms_norm":
            s["x"] = normal(shape, case["dtype"])
            s["residual"] = normal(shape, case["dtype"], 2.0) if case["residual"] else None
        else:
            s["h"] = normal(shape, case["dtype"], 2.0)
            s["dy"] = normal(shape, case["dtype"], 0.01)
            s["dh"] = normal(shape, case["dtype"], 0.01) if case["residual"] else None
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + 1e-6)
    elif op in ("preference", "preference_grad"):
        n, t, v = 2 * case["pairs"], case["length"], case["vocab"]
        s["logits"] = normal((n, t, v), case["dtype"], 2.0)
        s["labels"] = _labels(gen, case)
        ref = torch.zeros(n, dtype=torch.float64, device="cuda")
        for i in range(n):   # the reference model's log probabilities, near the policy's
            counted = s["labels"][i] >= 0
            rows = s["logits"][i][counted].float()
            at = s["labels"][i][counted]
            ref[i] = (rows.gather(1, at[:, None])[:, 0] - rows.logsumexp(1)).double().sum()
        noise = torch.randn(n, generator=gen, device="cuda")
        s["ref_logps"] = (ref + 5.0 * noise).float()
        s["dlosses"] = torch.full((case["pairs"],), 1.0 / case["pairs"], device="cuda")
    else:
        shapes = _adamw_shapes(case)
        s["grads"] = [normal(sh, case["grad"], 0.01) for sh in shapes]
        full = [normal(sh, "fp32", 0.02) for sh in shapes]
        s["params"] = [p.to(DT[case["dtype"]]) for p in full]
        s["masters"] = full if case["master"] else None
        s["exp_avgs"] = [normal(sh, case["state"], 0.003) for sh in shapes]
        s["exp_avg_sqs"] = [normal(sh, "fp32", 0.01).square().to(DT[case["state"]]) for sh in shapes]
        s["decays"] = [0.1 if len(sh) == 2 else 0.0 for sh in shapes]
    return s


# --------------------------------------------------------------------- run

BETA, EPS, LR, BETAS, STEP = 0.1, 1e-6, 3e-4, (0.9, 0.95), 1000
ADAM_EPS = 1e-8


def run(s):
    case = s["case"]
    return _OPS[case["op"]](s, case)


def _embedding(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        return nsmi.ns_embedding(s["table"], s["ids"], scale=case["scale"])
    return (s["table"][s["ids"]].float() * case["scale"]).to(s["table"].dtype)


def _embedding_grad(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        return nsmi.ns_embedding_grad(s["grad"], s["ids"], case["rows"], scale=case["scale"],
                                      out_dtype=DT[case["out"]], out=s["into"],
                                      accumulate=case["accumulate"])
    total = torch.zeros((case["rows"], case["dim"]), device="cuda")
    total.index_add_(0, s["ids"], s["grad"].float())
    total.mul_(case["scale"])
    if case["accumulate"]:
        return s["into"].copy_(total.add_(s["into"].float()))
    return total.to(DT[case["out"]])


def _rms_norm(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        if case["out"] == "e4m3":
            q, scales, h, rstd = nsmi.ns_rms_norm_fp8(s["x"], s["weight"], residual=s["residual"],
                                                      eps=EPS)
            return {"q": q, "scales": scales, "h": h, "rstd": rstd}
        y, h, rstd = nsmi.ns_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return {"y": y, "h": h, "rstd": rstd}
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)   # the norm is that of the stored sum
    wide = h.float()
    rstd = 1.0 / torch.sqrt(wide.square().mean(-1) + EPS)
    y = wide * rstd[:, None] * s["weight"].float()
    if case["out"] != "e4m3":
        return {"y": y.to(DT[case["out"]]), "h": h, "rstd": rstd}
    scales = y.abs().amax(-1) / E4M3_MAX
    q = (y / scales[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return {"q": q, "scales": scales, "h": h, "rstd": rstd}


def _rms_norm_grad(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        dx, dw = nsmi.ns_rms_norm_grad(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    dy, unit = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - unit * (g * unit).mean(-1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * unit).sum(0).to(s["weight"].dtype)}


def _preference(s, case, grad=False):
    if own:
        import newton_schulz_matrix_amd as nsmi
        out = nsmi.ns_preference_loss(s["logits"], s["labels"], s["ref_logps"], beta=BETA,
                                      label_smoothing=case["smoothing"])
        losses, margins, logps, lse = out
        if not grad:
            return {"losses": losses, "margins": margins, "logps": logps, "lse": lse}
        dlogits = nsmi.ns_preference_loss_grad(s["logits"], s["labels"], margins, lse, s["dlosses"],
                                               beta=BETA, label_smoothing=case["smoothing"])
        return {"losses": losses, "margins": margins, "dlogits": dlogits}
    logits, labels = s["logits"].float(), s["labels"]
    n, eps = case["pairs"], case["smoothing"]
    counted = labels >= 0
    at = labels.clamp(min=0)[..., None]
    top = logits.amax(-1)
    powers = torch.exp(logits - top[..., None])
    sums = powers.sum(-1)
    token = (logits.gather(-1, at)[..., 0] - top).double() - torch.log(sums.double())
    sequences = torch.where(counted, token, torch.zeros_like(token)).sum(-1)
    ratios = sequences - s["ref_logps"].double()
    margins = BETA * (ratios[:n] - ratios[n:])
    # -log sigmoid(m) = log(1 + exp(-m))
    above = torch.clamp(margins, min=0) + torch.log1p(torch.exp(-margins.abs()))   # -log sigmoid(-m)
    losses = (1 - eps) * (above - margins) + eps * above
    if not grad:
        lse = top.double() + torch.log(sums.double())
        return {"losses": losses.float(), "margins": margins.float(), "logps": sequences.float(),
                "lse": torch.where(counted, lse, torch.zeros_like(lse)).float()}
    slope = BETA * (torch.sigmoid(margins) - (1 - eps)) * s["dlosses"].double()
    slope = torch.cat([slope, -slope])[:, None] * counted
    dlogits = powers * (-(slope / sums.double()).float())[..., None]
    dlogits.scatter_add_(-1, at, slope.float()[..., None])
    return {"losses": losses.float(), "margins": margins.float(),
            "dlogits": dlogits.to(s["logits"].dtype)}


def _preference_grad(s, case):
    return _preference(s, case, grad=True)


def _adamw(s, case):
    masters = s["masters"]
    if own:
        import newton_schulz_matrix_amd as nsmi
        nsmi.ns_adamw_step(s["params"], s["grads"], s["exp_avgs"], s["exp_avg_sqs"], step=STEP, lr=LR,
                           betas=BETAS, eps=ADAM_EPS, weight_decays=s["decays"], masters=masters)
    else:
        wide = masters if masters is not None else s["params"]
        [_adamw_one(*row) for row in zip(s["params"], wide, s["grads"], s["exp_avgs"],
                                         s["exp_avg_sqs"], s["decays"])]
    out = {"params": s["params"], "exp_avgs": s["exp_avgs"], "exp_avg_sqs": s["exp_avg_sqs"]}
    if masters is not None:
        out["masters"] = masters
    return out


def _adamw_one(param, wide, grad, exp_avg, exp_avg_sq, decay):
    g, p = grad.float(), wide.float()
    m = exp_avg.float() * BETAS[0] + g * (1 - BETAS[0])
    v = exp_avg_sq.float() * BETAS[1] + g * g * (1 - BETAS[1])
    root = torch.sqrt(v / (1 - BETAS[1] ** STEP)) + ADAM_EPS
    p = p * (1 - LR * decay) - LR / (1 - BETAS[0] ** STEP) * m / root
    exp_avg.copy_(m)
    exp_avg_sq.copy_(v)
    wide.copy_(p)
    param.copy_(p)


_OPS = {"embedding": _embedding, "embedding_grad": _embedding_grad, "rms_norm": _rms_norm,
        "rms_norm_grad": _rms_norm_grad, "preference": _preference,
        "preference_grad": _preference_grad, "adamw": _adamw}


# --------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "embedding":
        n = case["tokens"] * case["dim"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 8 * case["tokens"], "flops": n}
    if op == "embedding_grad":
        n = case["tokens"] * case["dim"]
        # summed into a given gradient, only the tokens' rows are touched (all of them, at most)
        rows = case["rows"] if not case["accumulate"] else 2 * min(case["rows"], case["tokens"])
        return {"bytes": n * SIZE[case["dtype"]] + 8 * case["tokens"]
                + rows * case["dim"] * SIZE[case["out"]], "flops": 2 * n}
    if op in ("rms_norm", "rms_norm_grad"):
        n, e = case["rows"] * case["dim"], SIZE[case["dtype"]]
        if op == "rms_norm":
            moved = n * e * (3 if case["residual"] else 1) + n * SIZE.get(case["out"], 1)
            moved += case["rows"] * (8 if case["out"] == "e4m3" else 4) + case["dim"] * e
            return {"bytes": moved, "flops": 5 * n}
        moved = n * e * (4 if case["residual"] else 3) + case["rows"] * 4 + 2 * case["dim"] * e
        return {"bytes": moved, "flops": 10 * n}
    if op in ("preference", "preference_grad"):
        rows = 2 * case["pairs"] * case["length"]
        n = rows * case["vocab"]
        # about 2/3 of the rows count; the gradient's other rows are written as zeros
        read, wrote = 0.65 * n * SIZE[case["dtype"]], n * SIZE[case["dtype"]]
        if op == "preference":
            return {"bytes": read + 12 * rows, "flops": 4 * 0.65 * n}
        return {"bytes": read + wrote + 12 * rows, "flops": 7 * 0.65 * n}
    n = case["dim"] * (case["rows"] + case["gains"])
    moved = 2 * (SIZE[case["dtype"]] + 2 * SIZE[case["state"]]) + SIZE[case["grad"]]
    if case["master"]:   # the 16-bit copy is only written
        moved += 8 - SIZE[case["dtype"]]
    return {"bytes": n * moved, "flops": 14 * n}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op == "embedding":
        return s["table"].double().index_select(0, s["ids"]) * case["scale"]
    if op == "embedding_grad":
        ids, order = torch.sort(s["ids"], stable=True)
        tokens, counts = torch.unique_consecutive(ids, return_counts=True)
        out = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        begin = torch.cumsum(counts, 0) - counts
        ends = torch.cat([begin, begin.new_tensor([ids.numel()])])
        g = s["grad"].double()[order]
        out[tokens] = torch.segment_reduce(g, "sum", offsets=ends, axis=0) * case["scale"]
        return out + s["into"].double() if case["accumulate"] else out
    if op == "rms_norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        norm = (h.pow(2).sum(1) / case["dim"] + EPS).sqrt()
        y = h / norm[:, None] * s["weight"].double()
        if case["out"] != "e4m3":
            return {"y": y, "h": h, "rstd": 1 / norm}
        top = y.abs().max(1).values
        return {"q": y * (E4M3_MAX / top)[:, None], "scales": top / E4M3_MAX, "h": h, "rstd": 1 / norm}
    if op == "rms_norm_grad":
        h, r, w = s["h"].double(), s["rstd"].double()[:, None], s["weight"].double()
        dy = s["dy"].double()
        dot = torch.bmm((dy * w)[:, None, :], h[:, :, None])[:, 0]
        dx = dy * w * r - h * r ** 3 * dot / case["dim"]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": torch.mv((dy * h).t().contiguous(), r[:, 0])}
    if op in ("preference", "preference_grad"):
        return _exact_preference(s, case)
    b1, b2 = BETAS
    out = {"params": [], "exp_avgs": [], "exp_avg_sqs": [], "masters": []}
    for i, g in enumerate(t.double() for t in s["grads"]):
        m = s["exp_avgs"][i].double().lerp(g, 1 - b1)
        v = s["exp_avg_sqs"][i].double().lerp(g.pow(2), 1 - b2)
        p = (s["masters"] or s["params"])[i].double()
        p = p - LR * (s["decays"][i] * p + (m / (1 - b1 ** STEP))
                      / ((v / (1 - b2 ** STEP)).sqrt() + ADAM_EPS))
        for key, t in (("params", p), ("exp_avgs", m), ("exp_avg_sqs", v), ("masters", p)):
            out[key].append(t)
    if not case["master"]:
        del out["masters"]
    return out


def _exact_preference(s, case):
    n, t, v, b = 2 * case["pairs"], case["length"], case["vocab"], case["pairs"]
    lse = torch.zeros(n, t, dtype=torch.float64, device="cuda")
    logps = torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in range(n):   # one sequence at a time: 64 bits of all logits would be large
        counted = s["labels"][i] != IGNORED
        rows = s["logits"][i][counted].double()
        lse[i][counted] = rows.logsumexp(1)
        logps[i] = (rows.gather(1, s["labels"][i][counted][:, None])[:, 0]
                    - lse[i][counted]).sum()
    ref = s["ref_logps"].double()
    margins = BETA * ((logps[:b] - logps[b:]) - (ref[:b] - ref[b:]))
    log_sigmoid = torch.nn.functional.logsigmoid
    eps = case["smoothing"]
    losses = -(1 - eps) * log_sigmoid(margins) - eps * log_sigmoid(-margins)
    if case["op"] == "preference":
        return {"losses": losses, "margins": margins, "logps": logps, "lse": lse}
    slope = (-(1 - eps) * torch.sigmoid(-margins) + eps * torch.sigmoid(margins)) * BETA
    slope = slope * s["dlosses"].double()
    dlogits = torch.zeros(n, t, v, dtype=torch.float64, device="cuda")
    for i in range(n):
        counted = (s["labels"][i] != IGNORED).nonzero()[:, 0]
        k = slope[i] if i < b else -slope[i - b]
        d = torch.exp(s["logits"][i][counted].double() - lse[i][counted][:, None]) * -k
        at = s["labels"][i][counted]
        d[torch.arange(len(at), device="cuda"), at] += k
        dlogits[i][counted] = d
    return {"losses": losses, "margins": margins, "dlogits": dlogits}
