"""The operators around the recurrence, float64.  Test infrastructure only.

Each function is the definition, written per sequence with plain loops over
tokens.  ``scan`` also returns the size of the terms every output sums (the
recurrence run on absolute values), which the parity bars count roundings of.
"""
from __future__ import annotations

import numpy as np

from . import mamba2


def silu(v):
    v = np.asarray(v, np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, v / (1.0 + e), v * e / (1.0 + e))


def short_conv(x, weight, bias=None, history=None, act=True):
    """y[t] = act(bias + sum_k weight[:, k] x[t - K + 1 + k]) for one sequence.

    x [n, C]; weight [C, K]; history [K - 1, C] (the inputs before x; None: zeros).
    Returns (y [n, C], v [n, C] before the activation, size [n, C] = |bias| +
    sum |weight x|, the last K - 1 inputs)."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    C, K = weight.shape
    history = np.zeros((K - 1, C)) if history is None else np.asarray(history, np.float64)
    bias = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    every = np.concatenate([history, x])
    v = np.zeros((len(x), C))
    size = np.zeros((len(x), C))
    for t in range(len(x)):
        for k in range(K):
            v[t] += weight[:, k] * every[t + k]
            size[t] += np.abs(weight[:, k] * every[t + k])
    v, size = v + bias, size + np.abs(bias)
    return (silu(v) if act else v), v, size, every[len(every) - (K - 1):]


def scan(x, B, C, dt, A, D, S0=None):
    """The Mamba-2 recurrence over one sequence: x [n, H, P], B, C [n, G, N], dt [n, H].

    Returns (y [n, H, P], S [H, P, N] after the last token, size of y's terms, size of S's terms)."""
    n, H, P = x.shape
    S = np.zeros((H, P, B.shape[-1])) if S0 is None else np.asarray(S0, np.float64)
    Sa, A = np.abs(S), np.asarray(A, np.float64)
    y, size = np.zeros((n, H, P)), np.zeros((n, H, P))
    for t in range(n):
        S, y[t] = mamba2.step(S, x[t], B[t], C[t], dt[t], A, D)
        Sa, size[t] = mamba2.step(Sa, np.abs(x[t]), np.abs(B[t]), np.abs(C[t]), dt[t], A, np.abs(D))
    return y, S, size, Sa


def gated_norm(y, z, weight, group, eps, norm_first):
    """weight: one value a channel, or one a channel of a group."""
    y, z, weight = (np.asarray(a, np.float64) for a in (y, z, weight))
    T, C = y.shape
    w = np.tile(weight, C // weight.shape[0])
    h = (y if norm_first else y * silu(z)).reshape(T, C // group, group)
    h = (h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)).reshape(T, C) * w
    return h * silu(z) if norm_first else h


def accept(tokens, target, uniforms, draft=None, length=None):
    """One sequence: tokens [T], target [T + 1, V], draft [T, V] or None, uniforms [T + 1].

    Returns (accepted, next)."""
    T, V = len(tokens), target.shape[1]
    length = T if length is None else min(max(int(length), 0), T)
    p = np.asarray(target, np.float64)
    p = np.where(p > 0, p, 0.0)
    if draft is None:
        q = np.zeros((T, V))
        for i, x in enumerate(tokens):
            if 0 <= x < V:
                q[i, x] = np.inf  # a certain draft leaves its own token nothing
    else:
        q = np.asarray(draft, np.float64)
        q = np.where(q > 0, q, 0.0)
    a = 0
    while a < length:
        x = int(tokens[a])
        if not 0 <= x < V:
            break
        qx = 1.0 if draft is None else q[a, x]
        if not float(uniforms[a]) * qx < p[a, x]:
            break
        a += 1
    w = p[a]
    if a < length:
        rest = np.where(p[a] > q[a], p[a] - np.where(np.isfinite(q[a]), q[a], 0.0), 0.0)
        if rest.sum() > 0:
            w = rest
    if not w.sum() > 0:
        return a, -1
    run = np.cumsum(w)
    over = np.nonzero((run > float(uniforms[T]) * run[-1]) & (w > 0))[0]
    return a, int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])
