"""Plain fp64 reference of the calls around the module in the residual stream:
token embedding, residual sum with RMSNorm and E4M3 codes, gated feed-forward
block, and their backward passes.  numpy only, written from the formulas in
``include/engram.h``; the CPU tests pin the backward passes by differences.
"""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def embed(tok, E, scale=1.0):
    """scale * E[tok] per position; a zero row for an id outside the table."""
    tok = np.asarray(tok).reshape(-1)
    h = np.zeros((tok.size, E.shape[1]))
    for i, v in enumerate(tok):
        if 0 <= v < E.shape[0]:
            h[i] = scale * E[v]
    return h


def embed_grad(tok, d_h, V, scale=1.0):
    """(d_E, sum of magnitudes, occurrences): row v sums the rows of d_h whose token is v."""
    tok = np.asarray(tok).reshape(-1)
    d_E, mag, cnt = np.zeros((V, d_h.shape[1])), np.zeros((V, d_h.shape[1])), np.zeros(V, dtype=np.int64)
    for i, v in enumerate(tok):
        if 0 <= v < V:
            d_E[v] += scale * d_h[i]
            mag[v] += np.abs(scale * d_h[i])
            cnt[v] += 1
    return d_E, mag, cnt


def add_norm(x, res=None, gain=None, eps=1e-6):
    """(s, r, y): the sum, 1/rms per row, the normed rows."""
    s = x if res is None else x + res
    r = 1.0 / np.sqrt((s * s).mean(1) + eps)
    y = s * r[:, None]
    return s, r, y if gain is None else y * gain


def add_norm_grad(d_y, s, r, gain=None, d_sum=None):
    """(d_x, d_gain) with r as given (the forward's 1/rms)."""
    sh = s * r[:, None]
    t = d_y if gain is None else d_y * gain
    d_x = r[:, None] * (t - sh * (t * sh).mean(1, keepdims=True))
    return (d_x if d_sum is None else d_x + d_sum), (d_y * sh).sum(0)


def act(g, kind):
    """(act(g), act'(g)); GELU in its tanh form."""
    if kind == "silu":
        p = 1.0 / (1.0 + np.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def ffn(x, Wgu, Wd, kind, res=None):
    """(y, gu): y = (act(x Wg^T) * (x Wu^T)) Wd^T (+ res), gu = x [Wg; Wu]^T."""
    f = Wd.shape[1]
    gu = x @ Wgu.T
    y = (act(gu[:, :f], kind)[0] * gu[:, f:]) @ Wd.T
    return (y if res is None else y + res), gu


def ffn_grad(d_y, x, gu, Wgu, Wd, kind):
    """(d_x, d_Wgu, d_Wd)"""
    f = Wd.shape[1]
    a, da = act(gu[:, :f], kind)
    u = gu[:, f:]
    d_a = d_y @ Wd
    d_gu = np.concatenate([d_a * u * da, d_a * a], 1)
    return d_gu @ Wgu, d_gu.T @ x, d_y.T @ (a * u)
