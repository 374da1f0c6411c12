"""Plain 64-bit implementations (numpy) of the operators around the expert products, from their definitions."""
from __future__ import annotations

import numpy as np


def plan(ids, first, local, align, rows):
    """(offs, slot, src, dropped), pair by pair in order."""
    T, k = ids.shape
    pairs = [[] for _ in range(local)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if first <= e < first + local:
            pairs[e - first].append(p)
    offs, slot, src = np.zeros(local, np.int32), np.full(T * k, -1, np.int32), np.full(rows, -1, np.int32)
    start, dropped = 0, 0
    for e, mine in enumerate(pairs):
        for i, p in enumerate(mine):
            if start + i < rows:
                slot[p], src[start + i] = start + i, p
            else:
                dropped += 1
        start += (len(mine) + align - 1) // align * align
        offs[e] = min(start, rows)
    return offs, slot.reshape(T, k), src, dropped


def dispatch(x, src, k):
    out = np.zeros((len(src), x.shape[1]), x.dtype)
    here = src >= 0
    out[here] = x[src[here] // k]
    return out


def combine(y, weights, slot):
    """(out, sum of the terms' magnitudes); weights None: all one."""
    T, k = slot.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t, j in zip(*np.nonzero(slot >= 0)):
        term = y[slot[t, j]].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def combine_grad(dout, y, weights, slot, rows):
    """(dy, dweights, sum of the magnitudes of dweights' terms)"""
    T, k = slot.shape
    dy, dw, mag = np.zeros((rows, y.shape[1])), np.zeros((T, k)), np.zeros((T, k))
    for t, j in zip(*np.nonzero(slot >= 0)):
        d, r = dout[t].astype(np.float64), y[slot[t, j]].astype(np.float64)
        dy[slot[t, j]] = float(weights[t, j]) * d
        dw[t, j], mag[t, j] = d @ r, np.abs(d) @ np.abs(r)
    return dy, dw, mag


def norm(grads):
    return np.sqrt(sum(np.square(g.astype(np.float64)).sum() for g in grads))


def factor(norm, max_norm, eps=1e-6):
    return min(1.0, max_norm / (norm + eps))
