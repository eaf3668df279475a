"""Float64 oracle of the operators around the expert layer: scored routing,
the residual norm, the combine, and their gradients, from their definitions
in include/moe.h.  Plain loops where a loop says it best."""
from __future__ import annotations

from typing import Optional

import numpy as np


def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """Scores of every expert; a logit of -inf or NaN scores 0."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    out = np.zeros_like(l)
    if score == "sigmoid":
        pos = l >= 0
        out[pos] = 1.0 / (1.0 + np.exp(-l[pos]))
        out[~pos] = np.exp(l[~pos]) / (1.0 + np.exp(l[~pos]))
        return out
    for t, row in enumerate(l):
        top = row.max()
        if top == -np.inf:
            continue                                 # masked throughout
        if top == np.inf:
            e = (row == np.inf).astype(np.float64)
        else:
            e = np.exp(row - top)
        out[t] = e / e.sum()
    return out


def route_scored(logits, bias, k, score="softmax", groups=1, topk_groups=1,
                 group_top=1, renormalize=True, scale=1.0):
    """(ids [T][k], weights [T][k], counts [E])."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    s = scores(l, score)
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    per = E // groups
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        choice = {}                                  # the unmasked experts
        for e in range(E):
            c = s[t, e] + b[e]
            if not np.isnan(l[t, e]) and l[t, e] > -np.inf and c > -np.inf:
                choice[e] = c
        total = {}                                   # groups with one of them
        for g in range(groups):
            live = sorted((choice[e] for e in range(g * per, (g + 1) * per)
                           if e in choice), reverse=True)
            if live:
                total[g] = sum(live[:group_top])
        order = sorted(range(groups),
                       key=lambda g: (g not in total, -total.get(g, 0.0), g))
        kept = sorted(order[:topk_groups])
        cand = [e for g in kept for e in range(g * per, (g + 1) * per)]
        cand.sort(key=lambda e: (e not in choice, -choice.get(e, 0.0), e))
        ids[t] = cand[:k]
        w[t] = s[t, ids[t]]
        if renormalize:
            S = w[t].sum()
            w[t] = w[t] / S if S > 0 else 0.0
    counts = np.bincount(ids.reshape(-1), minlength=E).astype(np.int32)
    return ids, w * scale, counts


def route_scored_backward(logits, ids, d_w, score="softmax",
                          renormalize=True, scale=1.0):
    """d_logits [T][E]: through the Jacobian of the chosen weights, slot by
    slot."""
    s = scores(logits, score)
    T, E = s.shape
    k = ids.shape[1]
    out = np.zeros((T, E))
    for t in range(T):
        if score == "sigmoid":
            J = np.diag(s[t] * (1.0 - s[t]))         # ds / dl
            hot = np.asarray(logits[t], dtype=np.float64)
            for e in range(E):                       # 1 - s without cancelling
                if hot[e] > 0:
                    x = np.exp(-hot[e])
                    J[e, e] = s[t, e] * x / (1.0 + x)
        else:
            J = np.diag(s[t]) - np.outer(s[t], s[t])
        ch = s[t, ids[t]]
        if renormalize:
            S = ch.sum()
            if S == 0:
                continue
            W = (np.eye(k) - np.outer(ch / S, np.ones(k))) / S   # dw / ds
        else:
            W = np.eye(k)
        out[t] = scale * (np.asarray(d_w[t], dtype=np.float64) @ W @ J[ids[t]])
    return out


def unit(z: np.ndarray, eps: float) -> np.ndarray:
    return z / np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps)


def residual_norm(y, resid, post_gain, gate, pre_gain, eps=1e-6,
                  gain_offset=0.0, residual_scale=1.0):
    """(resid_out, x_out or None); every operand float64 or None."""
    r = np.array(resid, dtype=np.float64)
    if y is not None:
        v = np.asarray(y, dtype=np.float64)
        if post_gain is not None:
            v = unit(v, eps) * (gain_offset + post_gain)
        r = r + residual_scale * (v if gate is None else gate * v)
    x = None if pre_gain is None else unit(r, eps) * (gain_offset + pre_gain)
    return r, x


def unit_backward(z: np.ndarray, d: np.ndarray, eps: float) -> np.ndarray:
    """Gradient of unit: (d - u mean(d u)) / s with s the root and u = z/s."""
    s = np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps)
    u = z / s
    return (d - u * np.mean(d * u, axis=-1, keepdims=True)) / s


def residual_norm_backward(y, resid_out, post_gain, gate, pre_gain, d_x,
                           d_resid_out, eps=1e-6, gain_offset=0.0,
                           residual_scale=1.0) -> dict:
    out = {}
    r = resid_out
    g = 0.0 if d_resid_out is None else np.array(d_resid_out)
    if pre_gain is not None:
        out["d_pre"] = np.sum(d_x * unit(r, eps), axis=0)
        g = g + unit_backward(r, d_x * (gain_offset + pre_gain), eps)
    out["d_resid"] = g
    v = y
    if post_gain is not None:
        v = unit(y, eps) * (gain_offset + post_gain)
    if gate is not None:
        d = residual_scale * g * v
        out["d_gate"] = reduce_to(d, gate.shape)
    d_v = residual_scale * g * (1.0 if gate is None else gate)
    out["d_y"] = d_v
    if post_gain is not None:
        out["d_post"] = np.sum(d_v * unit(y, eps), axis=0)
        out["d_y"] = unit_backward(y, d_v * (gain_offset + post_gain), eps)
    return out


def reduce_to(d: np.ndarray, shape) -> np.ndarray:
    for axis in (0, 1):
        if shape[axis] == 1:
            d = d.sum(axis=axis, keepdims=True)
    return d


def combine_rows(y_perm, pair_row, w, y_shared: Optional[np.ndarray]):
    T, k = pair_row.shape
    out = np.zeros((T, y_perm.shape[1]))
    for t in range(T):
        for j in range(k):
            if pair_row[t, j] >= 0:
                out[t] += float(w[t, j]) * y_perm[pair_row[t, j]].astype(np.float64)
    return out if y_shared is None else out + y_shared


def combine_backward(d_out, y_perm, pair_row, w):
    """(d_y_perm with rows of no pair at NaN, d_topk_w)."""
    T, k = pair_row.shape
    d_y = np.full(y_perm.shape, np.nan)
    d_w = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            row = pair_row[t, j]
            if row >= 0:
                d_y[row] = float(w[t, j]) * d_out[t]
                d_w[t, j] = np.dot(d_out[t], y_perm[row].astype(np.float64))
    return d_y, d_w
