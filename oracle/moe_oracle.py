"""Plain fp64 CPU oracle of the operators that follow the attention in a decoder layer: the
residual stream's root-mean-square norm, the routing of tokens to experts ("DeepSeek-V4" doc,
MoE: sqrt(softplus) scores, e_score_correction_bias; "DeepSeek-V3.2" doc: sigmoid scores,
n_group / topk_group, norm_topk_prob) and the experts' clamped SwiGLU products.  One token at a
time, sharing no code with the CUDA library: test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np


def rms_norm(x, residual, weight, eps):
    """(r, y) with r = x + residual and y = r / sqrt(mean(r^2) + eps) * weight, row by row."""
    r = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    y = np.empty_like(r)
    w = np.asarray(weight, np.float64)
    for t in range(r.shape[0]):
        y[t] = r[t] / math.sqrt(float(np.dot(r[t], r[t])) / r.shape[1] + eps) * w
    return r, y


def group_scales(y, group=128, largest=448.0):
    """max |y| / 448 of every group of 128 consecutive channels (the last one may be shorter);
    1 for a group of zeros."""
    T, h = y.shape
    n = -(-h // group)
    s = np.empty((T, n))
    for g in range(n):
        s[:, g] = np.abs(y[:, g * group:(g + 1) * group]).max(axis=1) / largest
    s[s == 0] = 1.0
    return s


def score(fn, logits):
    """Scores of one token's experts."""
    l = np.asarray(logits, np.float64)
    if fn == "softmax":
        if np.all(l == -np.inf):
            return np.zeros_like(l)
        e = np.exp(l - l.max())
        return e / e.sum()
    if fn == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    return np.sqrt(np.log1p(np.exp(-np.abs(l))) + np.maximum(l, 0.0))


def route(logits, bias, *, fn, topk, n_group=1, topk_group=1, renorm=True, routed_scale=1.0):
    """(ids, weights): per token the topk experts of largest score + bias among the topk_group
    groups with the largest sum of their two best, in descending order, lower index first among
    equals; weights from the scores alone."""
    T, E = logits.shape
    per = E // n_group
    ids = np.empty((T, topk), np.int64)
    w = np.empty((T, topk))
    for t in range(T):
        s = score(fn, logits[t])
        c = s + (0 if bias is None else np.asarray(bias, np.float64))
        c = np.where(np.isnan(c), -np.inf, c)
        best = []
        for g in range(n_group):
            two = sorted(c[g * per:(g + 1) * per], reverse=True)[:2]
            best.append(sum(two))
        groups = sorted(range(n_group), key=lambda g: (-best[g], g))[:topk_group]
        cand = [e for e in range(E) if e // per in groups]
        chosen = sorted(cand, key=lambda e: (-c[e], e))[:topk]
        ids[t] = chosen
        w[t] = s[chosen]
        if renorm:
            w[t] = w[t] / (w[t].sum() + 1e-20)
    return ids, w * routed_scale


def expert_mlp(x, ids, weights, w13, w2, limit=0.0):
    """out[t] = sum_j weights[t,j] * W2_e (silu(min(g, L)) * clamp(u, -L, L)); ids outside the
    experts contribute nothing."""
    T, h = x.shape
    E, f = w13.shape[0], w13.shape[1] // 2
    out = np.zeros((T, h))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            a = w13[e].astype(np.float64) @ x[t].astype(np.float64)
            g, u = a[:f], a[f:]
            if limit > 0:
                g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
            out[t] += float(weights[t, j]) * (w2[e].astype(np.float64) @ (score("sigmoid", g) * g * u))
    return out
