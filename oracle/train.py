"""Float64 oracle of the 8-bit checkpoints and of the experts' forward and
backward pass, from their definitions in include/moe.h."""
from __future__ import annotations

import numpy as np

from . import fp8, moe


def checkpoint_scale(values) -> float:
    """The scale of one group: the smallest power of two from 2^-100 on that
    brings its finite values to 448 or less, 1 for a group of zeros."""
    size = np.abs(np.asarray(values, dtype=np.float64))
    size = size[np.isfinite(size)]
    top = float(size.max()) if size.size else 0.0
    if top == 0.0:
        return 1.0
    s = 2.0 ** -100
    while top / s > 448.0:
        s *= 2.0
    return s


def checkpoint(rows):
    """(codes [T][C], scales [T][ceil(C / 128)]) of rows [T][C]."""
    rows = np.asarray(rows, dtype=np.float64)
    T, C = rows.shape
    codes = np.zeros((T, C), dtype=np.uint8)
    scales = np.ones((T, -(-C // 128)), dtype=np.float32)
    for t in range(T):
        for n in range(scales.shape[1]):
            part = rows[t, 128 * n:128 * n + 128]
            s = checkpoint_scale(part)
            q = part / s
            if s == 2.0 ** 120:
                q = np.clip(q, -240.0, 240.0)
            fine = np.isfinite(q)
            c = fp8.e4m3_encode(np.where(fine, q, 0.0))
            codes[t, 128 * n:128 * n + part.size] = np.where(fine, c, 0x7F)
            scales[t, n] = s
    return codes, scales


def values(codes, scales):
    """What codes and scales stand for (the code of NaN is NaN)."""
    codes = np.asarray(codes)
    v = fp8.e4m3_decode(codes & 0x7F) * np.where(codes & 0x80, -1.0, 1.0)
    v = np.where((codes & 0x7F) == 0x7F, np.nan, v)
    s = np.repeat(np.asarray(scales, dtype=np.float64), 128, axis=1)
    return v * s[:, :codes.shape[1]]


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def expert_forward(x, wg, wu, wd, round_h=True):
    """(gate, up, y) of one expert on rows x."""
    g, u = x @ wg, x @ wu
    h = g * sigmoid(g) * u
    return g, u, (moe.round_to_bf16(h) if round_h else h) @ wd


def expert_backward(x, g, u, w, d, wg, wu, wd):
    """Gradients of sum(w * y * d) over rows with route weights w [n]: (d_x,
    d_w, d_wg, d_wu, d_wd), y the expert's output with the gate and up
    products g, u as they are given and nothing rounded."""
    q = sigmoid(g)
    e = d @ wd.T
    h = g * q * u
    d_w = (e * h).sum(1)
    e = e * w[:, None]
    dg = e * u * (q + g * q * (1.0 - q))
    du = e * g * q
    return (dg @ wg.T + du @ wu.T, d_w, x.T @ dg, x.T @ du,
            (h * w[:, None]).T @ d)


def few_layer(x, ids, w, begin, experts, here=None, shared=None):
    """The layer's output for rows x [T][H] with routes ids, w [T][k]; experts:
    (wg, wu, wd) of the local logical experts; here[t][j] False: that pair's
    replica is not held here."""
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if begin <= e < begin + len(experts) and (here is None or here[t][j]):
                y = expert_forward(x[t:t + 1], *experts[e - begin])[2]
                out[t] += w[t, j] * y[0]
    if shared is not None:
        out += expert_forward(x, *shared)[2]
    return out
