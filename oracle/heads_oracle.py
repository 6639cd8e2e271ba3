"""Plain fp64 forms of the operators on heads and of the token log probabilities
(test infrastructure): norm of queries and keys with their rotation, causal
attention over packed sequences, log probabilities with entropy and likeliest
entries, and their gradients, straight from the formulas.

Inputs are numpy arrays of any float type, read as fp64; nothing is rounded.
"""

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


# ------------------------------------- norm and rotation of queries and keys

def angles(positions, inv_freq, sections=None):
    """(tokens, pairs): the angle of each pair at each token."""
    positions = _f64(positions).reshape(-1, np.asarray(positions).shape[-1])
    pairs = len(inv_freq)
    axis = np.repeat(np.arange(len(positions)), sections if len(positions) > 1 else [pairs])
    return positions[axis].T * _f64(inv_freq)


def pair_columns(pairs, interleaved):
    """Columns of the first and second value of each pair."""
    i = np.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def rotate(x, angle, interleaved=False):
    """x (tokens, heads, dim) with its pairs turned by angle (tokens, pairs)."""
    x = _f64(x)
    a, b = pair_columns(angle.shape[1], interleaved)
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    return y


def qk_norm_rope(x, weight, angle, eps, interleaved=False):
    x = _f64(x)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * _f64(weight)
    return rotate(x, angle, interleaved)


def qk_norm_rope_grad(dy, x, weight, angle, eps, interleaved=False):
    """(dx, dweight or None)."""
    g = rotate(dy, -angle, interleaved)
    if weight is None:
        return g, None
    x = _f64(x)
    rstd = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n, gw = x * rstd, g * _f64(weight)
    return rstd * (gw - n * np.mean(gw * n, axis=-1, keepdims=True)), np.sum(g * n, axis=(0, 1))


# ---------------------------------------------------------------- attention

def _sequences(offsets):
    offsets = np.asarray(offsets)
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:]) if b > a]


def _scores(q, k, scale):
    s = scale * (q @ k.T)
    return np.where(np.tril(np.ones(s.shape, dtype=bool)), s, -np.inf)


def attention(q, k, v, offsets, scale):
    """(out, lse (heads, tokens), spread): spread is sum_j P |v_j|; rows in no sequence are 0."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    tokens, heads, _ = q.shape
    group = heads // k.shape[1]
    out, spread, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((heads, tokens))
    for a, b in _sequences(offsets):
        for h in range(heads):
            s = _scores(q[a:b, h], k[a:b, h // group], scale)
            top = s.max(axis=-1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(axis=-1, keepdims=True)
            lse[h, a:b] = (top + np.log(total))[:, 0]
            out[a:b, h] = (p / total) @ v[a:b, h // group]
            spread[a:b, h] = (p / total) @ np.abs(v[a:b, h // group])
    return out, lse, spread


def attention_grad(dout, q, k, v, out, lse, offsets, scale, rel=0.0, dp_err=0.0):
    """(dq, dk, dv) with P = exp(S - lse) and delta = dout . out from the given out and
    lse, and how far each may be off if every P is off by `rel` of itself and every
    dout . v - delta by dp_err * (sum of its terms' magnitudes)."""
    dout, q, k, v, out, lse = map(_f64, (dout, q, k, v, out, lse))
    group = q.shape[1] // k.shape[1]
    grads = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    slack = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    for a, b in _sequences(offsets):
        for h in range(q.shape[1]):
            g, qh, kh, vh = dout[a:b, h], q[a:b, h], k[a:b, h // group], v[a:b, h // group]
            p = np.exp(_scores(qh, kh, scale) - lse[h, a:b, None])
            delta = np.sum(g * out[a:b, h], axis=-1, keepdims=True)
            terms = np.abs(g) @ np.abs(vh).T + np.sum(np.abs(g * out[a:b, h]), axis=-1, keepdims=True)
            ds = scale * p * (g @ vh.T - delta)
            ds_off = rel * np.abs(ds) + scale * p * dp_err * terms
            grads[0][a:b, h] = ds @ kh
            grads[1][a:b, h // group] += ds.T @ qh
            grads[2][a:b, h // group] += p.T @ g
            slack[0][a:b, h] = ds_off @ np.abs(kh)
            slack[1][a:b, h // group] += ds_off.T @ np.abs(qh)
            slack[2][a:b, h // group] += rel * p.T @ np.abs(g)
    return grads, slack


# ---------------------------------------------------- token log probabilities

def token_logps(logits, tokens, top=0):
    """(logps, lse, entropy, top_logps, top_ids); rows whose token is not in the
    vocabulary are 0, and -1 in top_ids."""
    z, tokens = _f64(logits), np.asarray(tokens)
    vocab = z.shape[1]
    keep = (tokens >= 0) & (tokens < vocab)
    m = z.max(axis=-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        log_total = np.log(np.sum(np.exp(z - m), axis=-1, keepdims=True))
        lse = m + log_total
        logp = z - m - log_total      # (beside the lowest fp32 value lse no longer holds log_total)
        p = np.exp(logp)
        entropy = -np.sum(np.where(p > 0, p * logp, np.where(np.isnan(p), p, 0.0)), axis=-1)
    picked = np.take_along_axis(logp, np.where(keep, tokens, 0)[:, None], -1)[:, 0]
    # -0 equals 0; a NaN comes behind everything
    order = np.argsort(-np.where(np.isnan(z), -np.inf, z + 0.0), axis=-1, kind="stable")[:, :top]
    top_logps = np.where(keep[:, None], np.take_along_axis(logp, order, -1), 0.0)
    ids = np.where(keep[:, None], order, -1)
    return (np.where(keep, picked, 0.0), np.where(keep, lse[:, 0], 0.0), np.where(keep, entropy, 0.0),
            top_logps, ids)


def token_logps_grad(logits, tokens, lse, entropy, dlogps, dentropy=None):
    """Gradient for the given lse and entropy."""
    z, tokens = _f64(logits), np.asarray(tokens)
    keep = (tokens >= 0) & (tokens < z.shape[1])
    x = z - _f64(lse)[:, None]
    p = np.exp(x)
    d = -_f64(dlogps)[:, None] * p
    if dentropy is not None:
        with np.errstate(invalid="ignore"):
            d = d - np.where(p > 0, _f64(dentropy)[:, None] * p * (x + _f64(entropy)[:, None]), 0.0)
    at = np.where(keep, tokens, 0)
    d[np.arange(len(z)), at] += _f64(dlogps)
    return np.where(keep[:, None], d, 0.0)
