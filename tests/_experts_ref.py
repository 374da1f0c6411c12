"""Plain 64-bit implementations (numpy) of the expert-weight operators, written from their definitions, and input builders."""
from __future__ import annotations

import numpy as np


def bf16_round(x):
    """fp32 values nearest (ties to even) in bf16 to float64/float32 x (finite)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def e4m3_table():
    t = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = f / 8.0 * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        t[b] = -v if b & 128 else v
        if e == 15 and f == 7:
            t[b] = np.nan
    return t


def dequantise(q, s):
    """E4M3 bytes [..., n] and E8M0 bytes [..., n/32] -> float64."""
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return e4m3_table()[q] * np.repeat(scale, 32, axis=-1)


def choice_values(x, router, bias=None, score="softmax"):
    """(score, score + bias) [T, experts] in 64 bits."""
    logits = x.astype(np.float64) @ router.astype(np.float64).T
    if score == "softmax":
        p = np.exp(logits - logits.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-logits))
    return p, p if bias is None else p + bias.astype(np.float64)


def route(x, router, top_k, bias=None, score="softmax", renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k], gap [T]): the choice in 64 bits; gap is the smallest distance between the choice
    value of one of the first k + 1 experts and the next (how far the choice is from a tie)."""
    p, choice = choice_values(x, router, bias, score)
    order = np.argsort(-choice, axis=-1, kind="stable")
    ids = order[:, :top_k]
    w = np.take_along_axis(p, ids, -1)
    if renormalize:
        w = w / w.sum(-1, keepdims=True)
    first = np.take_along_axis(choice, order[:, :top_k + 1], -1)
    gap = np.min(first[:, :-1] - first[:, 1:], axis=-1) if first.shape[1] > 1 else np.full(len(x), np.inf)
    return ids, w * scale, gap


def moe_layer(x, w13, w2, ids, weights, first=0):
    """(y, absacc) in 64 bits from decoded weights w13 [local, 2 I, H], w2 [local, H, I] and a routing.
    absacc: sum over experts of weight * |W2| |h|, the scale of the last product's rounding errors."""
    T, H = x.shape
    local, I2, _ = w13.shape
    I = I2 // 2
    y, acc = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, w in zip(ids[t], weights[t]):
            if 0 <= e - first < local:
                gu = w13[e - first] @ x[t].astype(np.float64)
                h = gu[:I] / (1.0 + np.exp(-gu[:I])) * gu[I:]
                y[t] += w * (w2[e - first] @ h)
                acc[t] += abs(w) * np.sqrt(np.square(w2[e - first]) @ np.square(h))
    return y, acc


def muon(grad, momentum=None, mu=0.95, nesterov=True, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """(out, momentum') in 64 bits; grad [E, N, K]."""
    g = grad.astype(np.float64)
    m = None if momentum is None else mu * momentum.astype(np.float64) + g
    u = g if m is None else (g + mu * m if nesterov else m)
    a, b, c = coeffs
    out = np.empty_like(g)
    for e in range(len(g)):
        X = u[e] / (np.sqrt(np.square(u[e]).sum()) + eps)
        if X.shape[0] > X.shape[1]:
            X = X.T
        for _ in range(steps):
            A = X @ X.T
            X = a * X + (b * A + c * (A @ A)) @ X
        out[e] = X.T if g.shape[1] > g.shape[2] else X
    return out, m
