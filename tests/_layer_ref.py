"""A training step's layer (examples/layer_step.py) in 64 bits, with every quantisation and every rounding to bf16 where the
layer has it. ``change`` leaves one term out, for the tests of what such a comparison notices."""
from __future__ import annotations

import numpy as np

import oracle
import _experts_ref as X
import _step_ref as R

# (not among them: which values share a scale, as a power of two changes no rounding but where values underflow)
CHANGES = ("silu's second term", "gate's sigmoid in the up part", "weights in dy", "softmax's sum", "one expert's gradient", "second choice of a token")


def quantised(a):
    """What the E4M3 bytes and block scales of a's last axis stand for."""
    a = np.ascontiguousarray(a, dtype=np.float32)
    q, s = oracle.quantize_tokenwise(a.reshape(-1, a.shape[-1]))
    return X.dequantise(q, s).reshape(a.shape)


def rounded(a):
    return X.bf16_round(a).astype(np.float64)


def layer(x, dout, router, w13, w2, top_k, change=None):
    """(out, dx, dw13, dw2, drouter); x, dout: bf16 values [T, H]; router [E, H], w13 [E, 2 I, H], w2 [E, H, I]: fp32."""
    assert change is None or change in CHANGES
    E, I2, H = w13.shape
    I, T = I2 // 2, len(x)
    x, dout, router = (a.astype(np.float64) for a in (x, dout, router))
    logits = x @ router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    score = np.take_along_axis(logits, ids, 1)
    soft = np.exp(score - score.max(1, keepdims=True))
    soft /= soft.sum(1, keepdims=True)
    rows = (T * top_k + E * 31) // 32 * 32
    offs, slot, src, _ = R.plan(ids, 0, E, 32, rows)
    start = np.concatenate(([0], offs[:-1]))

    def grouped(a, w):
        out = np.zeros((rows, w.shape[1]))
        for e in range(E):
            out[start[e]:offs[e]] = a[start[e]:offs[e]] @ w[e].T
        return rounded(out)

    def contracted(a, b):
        """Blocks of 32 tokens share a scale."""
        qa, qb = quantised(a.T), quantised(b.T)
        out = np.stack([qa[:, start[e]:offs[e]] @ qb[:, start[e]:offs[e]].T for e in range(E)])
        if change == "one expert's gradient":
            out[E - 1] = 0
        return rounded(out)

    xs = R.dispatch(x, src, top_k)
    gu = grouped(quantised(xs), quantised(w13))
    g, u = gu[:, :I], gu[:, I:]
    sig = 1 / (1 + np.exp(-g))
    h = rounded(g * sig * u)
    y = grouped(quantised(h), quantised(w2))
    given = slot.copy()
    if change == "second choice of a token":
        given[7, 1] = -1
    out = rounded(R.combine(y, soft, given)[0])
    dy, dsoft, _ = R.combine_grad(dout, y, soft if change != "weights in dy" else np.ones_like(soft), slot, rows)
    dy = rounded(dy)
    dscore = soft * (dsoft - (0 if change == "softmax's sum" else (dsoft * soft).sum(1, keepdims=True)))
    drouter = np.zeros_like(router)
    np.add.at(drouter, ids.reshape(-1), dscore.reshape(-1)[:, None] * np.repeat(x, top_k, 0))
    dh = grouped(quantised(dy), quantised(np.swapaxes(w2, 1, 2)))
    dg = dh * u * sig * (1 + (0 if change == "silu's second term" else g * (1 - sig)))
    du = dh * g * (1 if change == "gate's sigmoid in the up part" else sig)
    dgu = rounded(np.concatenate((dg, du), 1))
    dxs = grouped(quantised(dgu), quantised(np.swapaxes(w13, 1, 2)))
    dx = rounded(R.combine(dxs, None, given)[0])
    return out, dx, contracted(dgu, xs), contracted(dy, h), drouter


def distance(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))
