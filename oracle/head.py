"""Float64 reference of the dense operators around the LittleBit layers: the
root-mean-square norm with its 8-bit output and its backward pass, the product
of 8-bit integers, and the token log probabilities with their gradient.

Written from the formulas, on float64 (or integer) arrays; what the GPU stores
in a narrower type in between (the rounded hidden state) is an input here.
"""

from __future__ import annotations

import numpy as np


def rmsnorm(h: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    h = np.asarray(h, np.float64)
    return h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rmsnorm_backward(dy, h, weight, eps, dhidden=None):
    """(dx, dweight)."""
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, weight))
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    u = w * dy
    dx = r * u - h * r ** 3 * np.mean(u * h, axis=1, keepdims=True)
    if dhidden is not None:
        dx = dx + np.asarray(dhidden, np.float64)
    return dx, np.sum(dy * h * r, axis=0)


def q8_scale(y: np.ndarray) -> np.ndarray:
    """One scale a row: its largest magnitude over 127."""
    return np.max(np.abs(np.asarray(y, np.float64)), axis=1) / 127.0


def q8_linear(xq, xscale, wq, wscale) -> np.ndarray:
    total = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T   # whole numbers below 2^53: exact
    return total * np.asarray(xscale, np.float64)[:, None] * np.asarray(wscale, np.float64)[None, :]


def max_and_logsum(x: np.ndarray):
    """(m, log sum exp(x - m)) of each row, m its maximum; (-infinity, -infinity) for a row of -infinity.  Kept
    apart: their sum may have no digits left for the second."""
    x = np.asarray(x, np.float64)
    m = np.max(x, axis=1, keepdims=True)
    at = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        return m[:, 0], np.log(np.sum(np.exp(x - at), axis=1))


def logsumexp(x: np.ndarray) -> np.ndarray:
    m, s = max_and_logsum(x)
    return m + s


def logprobs(x: np.ndarray):
    """(log p, entropy) of each row; a row of -infinity has log p -infinity and entropy 0."""
    x = np.asarray(x, np.float64)
    m, s = max_and_logsum(x)
    none = np.isneginf(s)[:, None]
    logp = np.where(none, -np.inf, x - np.where(none, 0.0, m[:, None]) - np.where(none, 0.0, s[:, None]))
    p = np.exp(logp)
    entropy = -np.sum(np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0), axis=1)
    return logp, entropy


def top(x: np.ndarray, k: int) -> np.ndarray:
    """Places of the k largest of each row, the lowest place first among equals, NaN before all."""
    x = np.asarray(x, np.float64)
    key = np.where(np.isnan(x), np.inf, x)
    return np.stack([np.lexsort((np.arange(x.shape[1]), -key[i], ~np.isnan(x[i])))[:k] for i in range(x.shape[0])])


def logprobs_backward(x, targets=None, dlogprob=None, dentropy=None, top_index=None, dtop=None) -> np.ndarray:
    x = np.asarray(x, np.float64)
    rows, vocab = x.shape
    logp, entropy = logprobs(x)
    p = np.exp(logp)
    g = np.zeros_like(x)                                  # gradient of every log probability
    if dlogprob is not None:
        for i, t in enumerate(targets):
            if t >= 0:
                g[i, t] += dlogprob[i]
    if dtop is not None:
        for i in range(rows):
            for j, t in enumerate(top_index[i]):
                g[i, t] += dtop[i][j]
    d = g - p * np.sum(g, axis=1, keepdims=True)
    if dentropy is not None:
        inner = np.where(p > 0, p * (np.where(p > 0, logp, 0.0) + entropy[:, None]), 0.0)
        d = d - np.asarray(dentropy, np.float64)[:, None] * inner
    d[np.isneginf(logsumexp(x))] = 0.0
    return d
