"""fp64 definitions of the operators around the training step (TEST INFRASTRUCTURE ONLY):
the scaled token-embedding lookup and the gradient of its table, layer norm and its
gradients, the global gradient norm and the clipped gradients. Inputs are the values the
GPU gets, as fp64; nothing here rounds.
"""
from __future__ import annotations

import numpy as np


def embed(ids, table, out, scale=1.0, token=None):
    """out with row i replaced by scale * table[ids[i]], zeros for an id outside the table;
    rows of `token` and rows past the ids stay."""
    got = np.array(out, np.float64)
    for i, t in enumerate(np.asarray(ids)):
        if token is not None and t == token:
            continue
        got[i] = scale * table[t] if 0 <= t < len(table) else 0.0
    return got


def embed_backward(ids, d_out, vocab, scale=1.0, token=None):
    """(gradient of the table, sum of |terms| of each of its elements)."""
    grad = np.zeros((vocab, d_out.shape[1]))
    mag = np.zeros_like(grad)
    ids = np.asarray(ids)
    keep = (ids >= 0) & (ids < vocab)
    if token is not None:
        keep &= ids != token
    np.add.at(grad, ids[keep], d_out[:len(ids)][keep])
    np.add.at(mag, ids[keep], np.abs(d_out[:len(ids)][keep]))
    return scale * grad, abs(scale) * mag


def layernorm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) over the last axis, biased variance."""
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    y = y if gamma is None else y * gamma
    return (y if beta is None else y + beta), mean, rstd


def layernorm_backward(x, mean, rstd, d_y, gamma=None):
    """(d_x, d_gamma, d_beta) for given statistics."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = d_y if gamma is None else d_y * gamma
    d_x = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return d_x, (d_y * xhat).sum(axis=0), d_y.sum(axis=0)


def clip_grads(grads, max_norm):
    """(norm, clipped gradients); infinities and NaN go through the formula."""
    with np.errstate(all="ignore"):
        norm = np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads)) if grads else np.float64(0.0)
        coef = np.float64(max_norm) / (norm + 1e-6)
        coef = np.float64(1.0) if coef >= 1.0 else coef
        return norm, [np.asarray(g, np.float64) * coef for g in grads]
