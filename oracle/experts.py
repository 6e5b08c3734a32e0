"""CPU oracle for routing and combining -- TEST INFRASTRUCTURE ONLY.

Binary64 throughout, one token at a time with Python loops; nothing here imports
the product package.
"""
from __future__ import annotations

import math

import numpy as np


def scores(logits, score: str) -> np.ndarray:
    """Softmax or sigmoid of one row; a row of -inf has softmax scores 0."""
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = np.max(l)
        e = np.exp(l - (0.0 if m == -math.inf else m))
        z = e.sum()
        return np.zeros_like(e) if z == 0 else e / z


def choose(logits, k: int, score: str, bias=None, groups: int = 1, top_groups: int | None = None):
    """(ids, the chosen scores) of one token."""
    s = scores(logits, score)
    b = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    b = np.where(np.isnan(b), -math.inf, b)
    E = len(b)
    if top_groups is not None and top_groups < groups:
        size = E // groups
        best = []
        for g in range(groups):
            part = sorted(b[g * size:(g + 1) * size], reverse=True)[:2]
            v = sum(part)
            best.append((-math.inf if math.isnan(v) else v))
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        b = np.array([b[e] if e // size in kept else -math.inf for e in range(E)])
    ids = sorted(range(E), key=lambda e: (-b[e], e))[:k]
    return np.array(ids), s[ids]


def weigh(s, renormalize: bool, scale: float) -> np.ndarray:
    if renormalize:
        z = s.sum()
        s = np.zeros_like(s) if z == 0 else s / z
    return s * scale


def route(logits, k, score, bias=None, groups=1, top_groups=None, renormalize=True, scale=1.0):
    """(weights, ids, offsets, tokens, slots) of all tokens."""
    T, E = np.shape(logits)
    ids, w = np.zeros((T, k), dtype=np.int64), np.zeros((T, k))
    for t in range(T):
        ids[t], s = choose(logits[t], k, score, bias, groups, top_groups)
        w[t] = weigh(s, renormalize, scale)
    order = sorted(range(T * k), key=lambda i: (ids.reshape(-1)[i], i))
    offsets = [0]
    for e in range(E):
        offsets.append(offsets[-1] + int((ids == e).sum()))
    slots = np.zeros(T * k, dtype=np.int64)
    slots[order] = np.arange(T * k)
    return w, ids, np.array(offsets), np.array([i // k for i in order]), slots.reshape(T, k)


def weights_at(logits, ids, score, renormalize, scale) -> np.ndarray:
    """The weights of one token's given choice, as a function of the logits."""
    return weigh(scores(logits, score)[ids], renormalize, scale)


def route_backward(dw, logits, ids, score, renormalize, scale) -> np.ndarray:
    """Gradients to the logits by the chain rule, written out."""
    T, E = np.shape(logits)
    out = np.zeros((T, E))
    for t in range(T):
        s = scores(logits[t], score)
        g = np.asarray(dw[t], dtype=np.float64) * scale
        c = ids[t]
        if renormalize:
            z = s[c].sum()
            g = np.zeros_like(g) if z == 0 else (g - (g * s[c]).sum() / z) / z
        ds = np.zeros(E)
        ds[c] = g
        out[t] = s * (ds - (ds * s).sum()) if score == "softmax" else ds * s * (1 - s)
    return out
