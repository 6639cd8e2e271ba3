"""Plain fp64 forms of the operators around the matrix update (test
infrastructure): embedding lookup, RMS norm with the residual's addition,
preference loss, AdamW, and their gradients, straight from the formulas.

Inputs are numpy arrays of any float type, read as fp64; nothing is rounded.
"""

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def embedding(table, ids, scale=1.0):
    """scale * table[ids]; ids outside the table give zeros."""
    table, ids = _f64(table), np.asarray(ids)
    inside = (ids >= 0) & (ids < len(table))
    return scale * table[np.where(inside, ids, 0)] * inside[..., None]


def embedding_grad(grad_out, ids, rows, scale=1.0, padding_idx=None):
    """(gradient, sum of the terms' magnitudes, number of terms of each row)."""
    g, ids = _f64(grad_out), np.asarray(ids).reshape(-1)
    g = g.reshape(len(ids), -1)
    keep = (ids >= 0) & (ids < rows)
    if padding_idx is not None:
        keep &= ids != padding_idx
    out, mag = np.zeros((rows, g.shape[1])), np.zeros((rows, g.shape[1]))
    np.add.at(out, ids[keep], scale * g[keep])
    np.add.at(mag, ids[keep], abs(scale) * np.abs(g[keep]))
    return out, mag, np.bincount(ids[keep], minlength=rows)


def rms_norm(h, weight, eps):
    """(y, rstd) of rows h."""
    h = _f64(h)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=-1) + eps)
    return h * rstd[..., None] * _f64(weight), rstd


def rms_norm_grad(dy, h, weight, eps, dh=None):
    """(dx, dweight)."""
    dy, h, w = _f64(dy), _f64(h), _f64(weight)
    _, rstd = rms_norm(h, w, eps)
    u, g = h * rstd[:, None], dy * w
    dx = rstd[:, None] * (g - u * np.mean(g * u, axis=-1, keepdims=True))
    if dh is not None:
        dx = dx + _f64(dh)
    return dx, np.sum(dy * u, axis=0)


def log_sigmoid(x):
    return np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    return np.exp(log_sigmoid(_f64(x)))


def _counted(labels, vocab):
    return (labels >= 0) & (labels < vocab)


def preference_loss(logits, labels, ref_logps, beta, smoothing):
    """(losses, margins, logps, lse); lse is 0 where a label does not count."""
    z, labels = _f64(logits), np.asarray(labels)
    b, vocab = z.shape[0] // 2, z.shape[2]
    keep = _counted(labels, vocab)
    top = z.max(axis=-1, initial=-np.inf)
    lse = top + np.log(np.sum(np.exp(z - top[..., None]), axis=-1))
    picked = np.take_along_axis(z, np.where(keep, labels, 0)[..., None], -1)[..., 0]
    logps = np.sum(np.where(keep, picked - lse, 0.0), axis=-1)
    ratio = logps - _f64(ref_logps)
    margins = beta * (ratio[:b] - ratio[b:])
    losses = -(1 - smoothing) * log_sigmoid(margins) - smoothing * log_sigmoid(-margins)
    return losses, margins, logps, np.where(keep, lse, 0.0)


def preference_loss_grad(logits, labels, ref_logps, dlosses, beta, smoothing):
    z, labels = _f64(logits), np.asarray(labels)
    _, margins, _, lse = preference_loss(z, labels, ref_logps, beta, smoothing)
    k = _f64(dlosses) * beta * (smoothing * sigmoid(margins) - (1 - smoothing) * sigmoid(-margins))
    k = np.concatenate([k, -k])[:, None, None]
    keep = _counted(labels, z.shape[2])
    onehot = np.zeros_like(z)
    np.put_along_axis(onehot, np.where(keep, labels, 0)[..., None], 1.0, -1)
    return np.where(keep[..., None], k * (onehot - np.exp(z - lse[..., None])), 0.0)


def adamw(w, g, m, v, step, lr, beta1, beta2, eps, decay):
    """(w, m, v) after one step."""
    w, g, m, v = _f64(w), _f64(g), _f64(m), _f64(v)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return w - lr * (decay * w + hat), m, v
