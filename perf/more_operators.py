"""Measured cases of the operators of a training step between its matrices: the
norm of each query's and key's head with the rotation of its positions and its
gradient, causal attention over packed sequences with grouped heads and its
gradient, and the log probabilities of given tokens with entropy and top
alternatives and their gradient.

``own`` selects the library's kernels; otherwise ``run`` computes the same
outputs with elementary torch operations in 32 bits (64 for angles), rounded
once at the end.

Real use of the cases. Queries, keys and values are parts of one projection's
output, (tokens, heads, head_dim). A batch is packed: sequences of different
lengths lie one behind the other, an int32 tensor of offsets says where each
begins, and rows behind the last one are padding, whose outputs are zeros.
Positions count within a sequence; with three axes (time, height, width) they
are those of a text with pictures in it. Logits have a few likely tokens in
each row, the given one often among them; a token of -100 does not count.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
IGNORED = -100
EPS = 1e-6
THETA = 500000.0
PACKED = "5113,2048,1,3329,777,0,2967,2021"   # 16256 tokens


def listed():
    return [
        # one new token for each of 4 served sequences: latency
        dict(name="head norm, 4 tokens", op="qk_norm", tokens=4, q_heads=32, k_heads=8, dim=128, rotary=128,
             axes=1, interleaved=False, norm=True, dtype="bf16", far=131072),
        # a training batch of packed sequences
        dict(name="head norm, 16384 tokens", op="qk_norm", tokens=16384, q_heads=32, k_heads=8, dim=128,
             rotary=128, axes=1, interleaved=False, norm=True, dtype="bf16", far=8192),
        # its backward pass
        dict(name="head norm gradient, 16384 tokens", op="qk_norm_grad", tokens=16384, q_heads=32, k_heads=8,
             dim=128, rotary=128, axes=1, interleaved=False, norm=True, dtype="bf16", far=8192),
        # text with pictures in full precision, few heads of an odd size, a part of each rotated
        dict(name="head norm gradient, 3 axes, fp32", op="qk_norm_grad", tokens=4099, q_heads=6, k_heads=2,
             dim=80, rotary=48, axes=3, interleaved=True, norm=True, dtype="fp32", far=2048),
        # one short prompt: latency
        dict(name="attention, 1 short prompt", op="attention", lengths="23", rest=0, q_heads=32, k_heads=8,
             dim=128, dtype="bf16"),
        # a training batch of sequences of different lengths, padded behind the last
        dict(name="attention, packed", op="attention", lengths=PACKED, rest=128, q_heads=32, k_heads=8,
             dim=128, dtype="bf16"),
        # one long document
        dict(name="attention, 1 long sequence", op="attention", lengths="16384", rest=0, q_heads=32, k_heads=8,
             dim=128, dtype="bf16"),
        # the backward pass of the training batch
        dict(name="attention gradient, packed", op="attention_grad", lengths=PACKED, rest=128, q_heads=32,
             k_heads=8, dim=128, dtype="bf16"),
        # a small model of odd sizes in fp16
        dict(name="attention gradient, odd, fp16", op="attention_grad", lengths="1031,333,97,1,602", rest=3,
             q_heads=6, k_heads=2, dim=80, dtype="fp16"),
        # the tokens that 8 served sequences have just taken, with 20 alternatives of each
        dict(name="log probabilities, 8 rows, top 20", op="logps", rows=8, vocab=50021, top=20, dtype="bf16"),
        # a reference model's pass over a training batch, with its 5 likeliest tokens
        dict(name="log probabilities, 4096 rows, top 5", op="logps", rows=4096, vocab=128000, top=5,
             dtype="bf16"),
        # a policy's step: gradient of its log probabilities and of an entropy bonus
        dict(name="log probability gradient, 4096 rows", op="logps_grad", rows=4096, vocab=128000, entropy=True,
             dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm", "qk_norm_grad", "attention", "attention", "attention_grad", "attention_grad",
                     "logps", "logps_grad"])
    if op in ("qk_norm", "qk_norm_grad"):
        dim = rng.choice([32, 64, 72, 80, 96, 128, 192, 256])
        k_heads = rng.choice([1, 2, 3, 4, 8])
        q_heads = k_heads * rng.choice([1, 2, 3, 4, 8])
        rotary = rng.choice([dim, dim, dim // 2 // 8 * 8])
        most = min(65536, (1 << 26) // (dim * (q_heads + k_heads)))
        return dict(op=op, tokens=_log_uniform(rng, 1, most), q_heads=q_heads, k_heads=k_heads, dim=dim,
                    rotary=rotary, axes=rng.choice([1, 1, 3]), interleaved=rng.random() < 0.3,
                    norm=rng.random() < 0.8, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    far=_log_uniform(rng, 256, 1 << 20))
    if op in ("attention", "attention_grad"):
        dim = rng.choice([16, 32, 64, 64, 72, 80, 96, 128, 128, 128])
        k_heads = rng.choice([1, 2, 3, 4, 8])
        q_heads = k_heads * rng.choice([1, 2, 3, 4, 8])
        longest = min(16384, int(math.sqrt((1 << 32) / q_heads)))
        one = _log_uniform(rng, 1, longest if op == "attention" else longest // 2)
        lengths = [one]
        while len(lengths) < 12 and rng.random() < 0.7:
            lengths.append(rng.choice([0, 1, rng.randint(1, one), rng.randint(1, one)]))
        while sum(x * x for x in lengths) * q_heads > 1 << 33 or sum(lengths) > 32768:
            lengths.pop()
        rng.shuffle(lengths)
        return dict(op=op, lengths=",".join(map(str, lengths)), rest=rng.choice([0, 0, 1, 61]), q_heads=q_heads,
                    k_heads=k_heads, dim=dim, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    vocab = _log_uniform(rng, 1000, 131072)
    case = dict(op=op, rows=_log_uniform(rng, 1, min(16384, (1 << 28) // vocab)), vocab=vocab)
    if op == "logps":
        case["top"] = rng.choice([0, 1, 5, 20])
    else:
        case["entropy"] = rng.random() < 0.5
    case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return case


# ------------------------------------------------------------------- inputs

def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def sections(case):
    """Pairs of a head that turn with each axis: half with time, the rest with height and width."""
    pairs = case["rotary"] // 2
    return [pairs] if case["axes"] == 1 else [pairs - 2 * (pairs // 4), pairs // 4, pairs // 4]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, scale=1.0, mean=0.0):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(mean).to(DT[dtype])

    op, s = case["op"], {"case": case}
    if op in ("qk_norm", "qk_norm_grad"):
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        qkv = normal((t, hq + 2 * hk, d), case["dtype"], 1.5)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"] = normal((d,), case["dtype"], 0.1, 1.0) if case["norm"] else None
        s["k_weight"] = normal((d,), case["dtype"], 0.1, 1.0) if case["norm"] else None
        s["inv_freq"] = (THETA ** (-torch.arange(0, case["rotary"], 2, dtype=torch.float64)
                                   / max(case["rotary"], 1))).float().cuda()
        # a packed batch: positions rise within a sequence, each begins somewhere
        step = torch.arange(t, device="cuda")
        begin = torch.randint(0, case["far"], (case["axes"], 1), generator=gen, device="cuda")
        s["positions"] = (begin + step) % case["far"]
        if case["axes"] == 1:
            s["positions"] = s["positions"][0]
        s["sections"] = sections(case) if case["axes"] > 1 else None
        if op == "qk_norm_grad":
            dqkv = normal((t, hq + 2 * hk, d), case["dtype"], 0.01)
            s["dq"], s["dk"] = dqkv[:, :hq], dqkv[:, hq:hq + hk]
    elif op in ("attention", "attention_grad"):
        lengths, hq, hk, d = _lengths(case), case["q_heads"], case["k_heads"], case["dim"]
        t = sum(lengths) + case["rest"]
        qkv = normal((t, hq + 2 * hk, d), case["dtype"])
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q"] *= 1.5   # some attention is peaked
        s["lengths"] = lengths
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        if op == "attention_grad":
            s["dout"] = normal((t, hq, d), case["dtype"], 0.01)
            s["out"], s["lse"] = _plain_attention(s, case)
    else:
        n, v = case["rows"], case["vocab"]
        s["logits"] = normal((n, v), case["dtype"], 2.5)
        s["tokens"] = torch.randint(0, v, (n,), generator=gen, device="cuda")
        row = torch.arange(n, device="cuda")
        s["logits"][row, s["tokens"]] += (8.0 * torch.rand(n, generator=gen, device="cuda")).to(DT[case["dtype"]])
        if n > 16:   # a prompt and what stands behind the end
            s["tokens"][torch.rand(n, generator=gen, device="cuda") < 0.2] = IGNORED
        if op == "logps_grad":
            logits, counted = s["logits"].float(), s["tokens"] >= 0
            lse = torch.logsumexp(logits, -1)
            p = torch.exp(logits - lse[:, None])
            entropy = lse - (p * logits).sum(-1)
            s["lse"], s["entropy"] = lse * counted, entropy * counted
            s["dlogps"] = torch.randn(n, generator=gen, device="cuda") / n
            s["dentropy"] = torch.full((n,), -0.01 / n, device="cuda") if case["entropy"] else None
    return s


# --------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    return _OPS[case["op"]](s, case)


def _angles(s, case):
    """cos and sin (tokens, 1, rotary / 2) of each pair's angle."""
    positions = s["positions"].double().reshape(case["axes"], -1)
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"),
                                   torch.tensor(sections(case), device="cuda"))
    angle = (positions[axis] * s["inv_freq"].double()[:, None]).t()[:, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turned(x, cos, sin, case, sign=1.0):
    """x (tokens, heads, dim) with its first `rotary` values turned in pairs."""
    r = case["rotary"]
    if case["interleaved"]:
        a, b = x[..., :r:2], x[..., 1:r:2]
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
    y = x.clone()
    first, second = a * cos - b * sin * sign, b * cos + a * sin * sign
    if case["interleaved"]:
        y[..., :r:2], y[..., 1:r:2] = first, second
    else:
        y[..., :r // 2], y[..., r // 2:r] = first, second
    return y


def _qk_norm(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        q, k = nsmi.ns_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"],
                                    eps=EPS, sections=s["sections"], interleaved=case["interleaved"])
        return {"q": q, "k": k}
    cos, sin = _angles(s, case)
    return {"q": _plain_head(s["q"], s["q_weight"], cos, sin, case),
            "k": _plain_head(s["k"], s["k_weight"], cos, sin, case)}


def _plain_head(x, weight, cos, sin, case):
    y = x.float()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    return _turned(y, cos, sin, case).to(x.dtype)


def _qk_norm_grad(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        dq, dk, dqw, dkw = nsmi.ns_qk_norm_rope_grad(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"],
                                                     s["k_weight"], s["positions"], s["inv_freq"], eps=EPS,
                                                     sections=s["sections"], interleaved=case["interleaved"])
    else:
        cos, sin = _angles(s, case)
        dq, dqw = _plain_head_grad(s["dq"], s["q"], s["q_weight"], cos, sin, case)
        dk, dkw = _plain_head_grad(s["dk"], s["k"], s["k_weight"], cos, sin, case)
    out = {"dq": dq, "dk": dk}
    if case["norm"]:
        out.update(dq_weight=dqw, dk_weight=dkw)
    return out


def _plain_head_grad(dy, x, weight, cos, sin, case):
    g = _turned(dy.float(), cos, sin, case, sign=-1.0)
    if weight is None:
        return g.to(x.dtype), None
    wide = x.float()
    rstd = 1.0 / torch.sqrt(wide.square().mean(-1, keepdim=True) + EPS)
    unit = wide * rstd
    dw = (g * unit).sum((0, 1)).to(weight.dtype)
    g = g * weight.float()
    return ((g - unit * (g * unit).mean(-1, keepdim=True)) * rstd).to(x.dtype), dw


def _by_head(x, at, n, groups):
    """Rows at .. at + n of x (tokens, heads, dim) as (k_heads, heads of a group * n, dim) in 32 bits."""
    h, d = x.shape[1:]
    return x[at:at + n].float().transpose(0, 1).reshape(h // groups, groups * n, d)


def _hidden(n, groups):
    """(groups * n, n): whether key j lies behind query i."""
    i = torch.arange(n, device="cuda")
    return (i[None, :] > i[:, None]).repeat(groups, 1)


def _plain_attention(s, case):
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    g, at = hq // hk, 0
    out = torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    lse = torch.zeros((hq, s["q"].shape[0]), device="cuda")
    for n in s["lengths"]:   # each sequence sees itself alone
        if n:
            q, k, v = _by_head(s["q"], at, n, g), _by_head(s["k"], at, n, 1), _by_head(s["v"], at, n, 1)
            p = torch.matmul(q, k.transpose(1, 2).contiguous()).mul_(d ** -0.5)
            p.masked_fill_(_hidden(n, g), -math.inf)
            top = p.amax(-1, keepdim=True)
            p.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v) / total
            out[at:at + n] = o.view(hq, n, d).transpose(0, 1).to(out.dtype)
            lse[:, at:at + n] = (top + torch.log(total)).view(hq, n)
        at += n
    return out, lse


def _attention(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        out, lse = nsmi.ns_attention(s["q"], s["k"], s["v"], s["offsets"])
    else:
        out, lse = _plain_attention(s, case)
    return {"out": out, "lse": lse}


def _attention_grad(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        dq, dk, dv = nsmi.ns_attention_grad(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["offsets"])
        return {"dq": dq, "dk": dk, "dv": dv}
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    g, at, scale = hq // hk, 0, d ** -0.5
    dq, dk, dv = (torch.zeros(s[x].shape, dtype=s[x].dtype, device="cuda") for x in ("q", "k", "v"))
    for n in s["lengths"]:
        if n:
            q, k, v = _by_head(s["q"], at, n, g), _by_head(s["k"], at, n, 1), _by_head(s["v"], at, n, 1)
            do, o = _by_head(s["dout"], at, n, g), _by_head(s["out"], at, n, g)
            lse = s["lse"][:, at:at + n].reshape(hk, g * n, 1)
            p = torch.matmul(q, k.transpose(1, 2).contiguous()).mul_(scale).sub_(lse).exp_()
            p.masked_fill_(_hidden(n, g), 0.0)
            dv[at:at + n] = torch.matmul(p.transpose(1, 2), do).transpose(0, 1).to(dv.dtype)
            ds = torch.matmul(do, v.transpose(1, 2).contiguous())
            ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            dk[at:at + n] = torch.matmul(ds.transpose(1, 2), q).transpose(0, 1).to(dk.dtype)
            dq[at:at + n] = torch.matmul(ds, k).view(hq, n, d).transpose(0, 1).to(dq.dtype)
        at += n
    return {"dq": dq, "dk": dk, "dv": dv}


def _logps(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        out = nsmi.ns_token_logps(s["logits"], s["tokens"], top=case["top"])
        logps, lse, entropy, top_logps, top_ids = out
    else:
        counted = s["tokens"] >= 0
        logits = s["logits"].float()
        top = logits.amax(-1, keepdim=True)
        x = logits - top
        powers = torch.exp(x)
        total = powers.sum(-1)
        log_total = torch.log(total)
        lse = (top[:, 0] + log_total) * counted
        entropy = (log_total - (powers * x).sum(-1) / total) * counted
        logps = (x.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0] - log_total) * counted
        if case["top"]:
            # one whole number for each entry, in the order of (value, lowest index first)
            bits = (logits + 0.0).view(torch.int32).long()
            key = torch.where(bits < 0, bits ^ 0x7fffffff, bits) * (1 << 24) + (case["vocab"] - torch.arange(
                case["vocab"], device="cuda"))
            top_ids = case["vocab"] - (key.topk(case["top"], -1).values & 0xffffff)
            top_logps = (x.gather(1, top_ids) - log_total[:, None]) * counted[:, None]
            top_ids = torch.where(counted[:, None], top_ids, -torch.ones_like(top_ids))
    out = {"logps": logps, "lse": lse, "entropy": entropy}
    if case["top"]:
        out.update(top_logps=top_logps, top_ids=top_ids)
    return out


def _logps_grad(s, case):
    if own:
        import newton_schulz_matrix_amd as nsmi
        return nsmi.ns_token_logps_grad(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogps"],
                                        dentropy=s["dentropy"])
    counted = (s["tokens"] >= 0)[:, None]
    x = s["logits"].float() - s["lse"][:, None]
    p = torch.exp(x)
    dlogps = s["dlogps"][:, None]
    d = -dlogps * p
    if case["entropy"]:
        d -= s["dentropy"][:, None] * p * (x + s["entropy"][:, None])
    d.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], dlogps)
    return torch.where(counted, d, torch.zeros_like(d)).to(s["logits"].dtype)


_OPS = {"qk_norm": _qk_norm, "qk_norm_grad": _qk_norm_grad, "attention": _attention,
        "attention_grad": _attention_grad, "logps": _logps, "logps_grad": _logps_grad}


# --------------------------------------------------------------------- work

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("qk_norm", "qk_norm_grad"):
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        less = 8 * case["axes"] * case["tokens"] + 2 * case["rotary"] + 2 * case["dim"] * e
        if op == "qk_norm":
            return {"bytes": 2 * n * e + less, "flops": 8 * n}
        # without the norm the gradient is a rotation of what arrives
        return {"bytes": (3 if case["norm"] else 2) * n * e + less, "flops": 14 * n}
    if op in ("attention", "attention_grad"):
        t, hq, hk, d = sum(_lengths(case)) + case["rest"], case["q_heads"], case["k_heads"], case["dim"]
        pairs = sum(n * (n + 1) // 2 for n in _lengths(case)) * hq
        if op == "attention":
            return {"bytes": t * d * e * 2 * (hq + hk) + 4 * hq * t, "flops": 4 * d * pairs}
        return {"bytes": t * d * e * 4 * (hq + hk) + 4 * hq * t, "flops": 10 * d * pairs}
    rows = case["rows"] * (0.8 if case["rows"] > 16 else 1.0)   # those that count
    n = rows * case["vocab"]
    if op == "logps":
        return {"bytes": n * e + case["rows"] * (20 + 12 * case["top"]), "flops": 6 * n}
    return {"bytes": n * e + case["rows"] * (case["vocab"] * e + 24), "flops": (8 if case["entropy"] else 5) * n}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op in ("qk_norm", "qk_norm_grad"):
        return _exact_heads(s, case)
    if op in ("attention", "attention_grad"):
        return _exact_attention(s, case)
    z, counted = s["logits"].double(), s["tokens"] != IGNORED
    logp = torch.log_softmax(z, -1)
    at = s["tokens"].where(counted, torch.zeros_like(s["tokens"]))[:, None]
    entropy = -torch.special.xlogy(torch.exp(logp), torch.exp(logp)).sum(-1)
    keep = counted.double()
    if op == "logps":
        out = {"logps": logp.gather(1, at)[:, 0] * keep, "lse": torch.logsumexp(z, -1) * keep,
               "entropy": entropy * keep}
        if case["top"]:
            out.update(top_logps=logp.topk(case["top"], -1).values * keep[:, None], top_ids=None)
        return out
    g = s["dlogps"].double()[:, None]
    d = -torch.softmax(z, -1) * g
    d[torch.arange(len(z), device="cuda"), at[:, 0]] += g[:, 0]
    if case["entropy"]:
        d -= s["dentropy"].double()[:, None] * torch.exp(logp) * (logp + entropy[:, None])
    return d * keep[:, None]


def _exact_heads(s, case):
    pairs, parts = case["rotary"] // 2, sections(case)
    positions = s["positions"].double().view(case["axes"], -1)
    begin, columns = 0, []
    for axis, width in enumerate(parts):
        columns.append(torch.outer(positions[axis], s["inv_freq"][begin:begin + width].double()))
        begin += width
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.cat(columns, 1))[:, None]

    def spin(x, by):
        head, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (pairs, 2)).contiguous()) * by
            return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)
        z = torch.complex(head[..., :pairs].contiguous(), head[..., pairs:].contiguous()) * by
        return torch.cat([z.real, z.imag, rest], -1)

    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"]
        rms = (x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
        if case["op"] == "qk_norm":
            out[name] = spin(x if w is None else x / rms * w.double(), turn)
            continue
        g = spin(s["d" + name].double(), turn.conj())
        if w is None:
            out["d" + name] = g
            continue
        out["d" + name + "_weight"] = (g * x / rms).flatten(0, 1).sum(0)
        g = g * w.double()
        out["d" + name] = g / rms - x * (g * x).sum(-1, keepdim=True) / (case["dim"] * rms ** 3)
    return out


def _exact_attention(s, case):
    hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
    wide = dict(dtype=torch.float64, device="cuda")
    names = ("q", "k", "v")
    out = torch.zeros(s["q"].shape, **wide)
    lse = torch.zeros((hq, len(out)), **wide)
    grads = [torch.zeros(s[x].shape, **wide) for x in names]
    ends = s["offsets"].tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        if a == b:
            continue
        seen = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").tril()
        for h in range(hq):
            q, k, v = (s[x][a:b, h if x == "q" else h * hk // hq].double() for x in names)
            scores = (q @ k.t() / math.sqrt(d)).where(seen, torch.tensor(-math.inf, **wide))
            p = torch.softmax(scores, -1)
            if case["op"] == "attention":
                out[a:b, h] = p @ v
                lse[h, a:b] = torch.logsumexp(scores, -1)
                continue
            do = s["dout"][a:b, h].double()
            dp = do @ v.t()
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
            grads[0][a:b, h] = ds @ k
            grads[1][a:b, h * hk // hq] += ds.t() @ q
            grads[2][a:b, h * hk // hq] += p.t() @ do
    if case["op"] == "attention":
        return {"out": out, "lse": lse}
    return dict(zip(("dq", "dk", "dv"), grads))
