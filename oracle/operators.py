"""The gate, layer norm and gradient clipping in plain numpy float64 -- TEST
INFRASTRUCTURE ONLY.

Written from the formulas in include/moe.h, row by row; inputs are float64
arrays holding the values of the float32 or bf16 inputs, outputs are unrounded.
It shares no code with the HIP library and never imports it.
"""
from __future__ import annotations

import math

import numpy as np

MASK_BELOW = -1e38
F32_MAX = float(np.finfo(np.float32).max)


def _row_scores(row, score):
    """Live experts (unmasked), logits with +inf at the largest float, scores."""
    live = np.array([not math.isnan(v) and v > MASK_BELOW for v in row])
    lg = np.array([min(v, F32_MAX) if ok else -math.inf for v, ok in zip(row, live)])
    s = np.zeros(len(row))
    if not live.any():
        return live, lg, s
    if score == "softmax":
        e = np.exp(lg - lg.max())
        s = e / e.sum()
    else:
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-lg[live]))
    return live, lg, s


def gate_row(row, k, score="softmax", bias=None, n_groups=1, keep_groups=None, group_score="max", renorm=True,
             scale=1.0):
    E = len(row)
    size = E // n_groups
    keep = n_groups if keep_groups is None else keep_groups
    live, lg, s = _row_scores(row, score)
    biased = s if bias is None else s + bias
    place = lg if bias is None else biased
    # a group's score, over its live experts
    best = []
    for g in range(n_groups):
        mine = [e for e in range(g * size, (g + 1) * size) if live[e]]
        if group_score == "max":
            best.append(max((place[e] for e in mine), default=-math.inf))
        else:
            best.append(sum(sorted((biased[e] for e in mine), reverse=True)[:2]) if mine else -math.inf)
    groups = sorted(range(n_groups), key=lambda g: (-best[g], g))[:keep]
    some = [e for e in range(E) if e // size in groups]
    some.sort(key=lambda e: (0, -place[e], e) if live[e] else (1, 0.0, e))
    idx = np.array(some[:k])
    if renorm:
        # ratios of scores, where they all underflow too
        on = [e for e in idx if live[e]]
        w = np.zeros(k)
        if on:
            if score == "softmax":
                top = max(lg[e] for e in on)
                part = {e: math.exp(lg[e] - top) for e in on}
            else:
                logs = {e: -math.log1p(math.exp(-lg[e])) if lg[e] > -30 else lg[e] - math.log1p(math.exp(lg[e]))
                        for e in on}
                top = max(logs.values())
                part = {e: math.exp(v - top) for e, v in logs.items()}
            w = np.array([part.get(e, 0.0) for e in idx]) / sum(part.values())
    else:
        w = s[idx]
    return idx, scale * w


def gate(logits, k, **kw):
    rows = [gate_row(r, k, **kw) for r in logits]
    return np.array([r[0] for r in rows], np.int32).reshape(-1, k), np.array([r[1] for r in rows]).reshape(-1, k)


def gate_backward(logits, idx, d_w, score="softmax", renorm=True, scale=1.0):
    """d_logits by the chain rule through w_i = scale s_i / sum s (renorm) or scale s_i."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        live, lg, s = _row_scores(logits[t], score)
        slots = [(int(e), float(g)) for e, g in zip(idx[t], d_w[t]) if 0 <= e < E and live[e]]
        d_s = np.zeros(E)
        if renorm:
            total = sum(s[e] for e, _ in slots)
            for e, g in slots:
                d_s[e] += scale * g / total
                for f, _ in slots:
                    d_s[f] -= scale * g * s[e] / total ** 2
        else:
            for e, g in slots:
                d_s[e] += scale * g
        if score == "softmax":
            out[t] = s * (d_s - float(d_s @ s))
        else:
            out[t] = d_s * s * (1.0 - s)
    return out


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    mean = x.mean(1, keepdims=True)
    hat = (x - mean) / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    return hat * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)


def layer_norm_backward(d_y, x, weight=None, eps=1e-5, d_skip=None):
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    hat = (x - mean) * rstd
    g = d_y if weight is None else d_y * weight
    d_x = rstd * (g - g.mean(1, keepdims=True) - hat * (g * hat).mean(1, keepdims=True))
    return dict(d_x=d_x if d_skip is None else d_x + d_skip, d_weight=(d_y * hat).sum(0), d_bias=d_y.sum(0))


def clip(grads, max_norm, eps=1e-6):
    norm = math.sqrt(sum(math.fsum((g.reshape(-1) ** 2).tolist()) for g in grads))
    factor = min(1.0, max_norm / (norm + eps))
    return norm, [g * factor for g in grads]
