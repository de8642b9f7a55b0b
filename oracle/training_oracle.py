"""CPU oracle of the operators around the layer in a training step (test infrastructure).

Only the tests import it; it shares no code with the CUDA library.  Plain numpy in
float64; where a definition names a float32 rounding (the 8-bit AdamW state and the
moments that lead to it, the embedding rows) the rounding is applied to the float64
value, which is exact for the product, quotient, sum and root of two float32 values
(53 >= 2 * 24 + 2 bits, so rounding twice equals rounding once).
"""
from __future__ import annotations

import math

import numpy as np

BLOCK8 = 256


def rn32(x):
    """The float32 rounding of float64 values, as float64."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def _blocks(x):
    """[ceil(n / 256), 256] with zeros past the end."""
    x = np.asarray(x, np.float64).reshape(-1)
    out = np.zeros((-(-x.size // BLOCK8), BLOCK8))
    out.reshape(-1)[:x.size] = x
    return out


def adam8_encode(x, top: int):
    """(k, d) of the values x: d = RN(max |x| / top^2) per block of 256, |k| the number of
    j >= 0 with RN(|x| RN(1 / d)) > j^2 + j + 1/2.  A block with a non-finite value: d = NaN,
    k = 0; d below 2^-126: d = 0, k = 0."""
    n = np.asarray(x).size
    b = _blocks(x)
    k, d = np.zeros(b.shape, np.int64), np.zeros(b.shape[0], np.float32)
    j = np.arange(top, dtype=np.float64)
    border = j * j + j + 0.5
    for i, row in enumerate(b):
        if not np.isfinite(row).all():
            d[i] = np.nan
            continue
        step = rn32(np.abs(row).max() / (top * top))
        if step < 2.0 ** -126:
            continue
        y = rn32(np.abs(row) * rn32(1.0 / step))
        k[i] = (y[:, None] > border).sum(axis=1) * np.where(row < 0, -1, 1)
        d[i] = np.float32(step)
    return k.reshape(-1)[:n], d


def adam8_decode(k, d):
    """k |k| d in float32 (as float64): RN(RN(k |k|) d)."""
    k = np.asarray(k, np.float64)
    step = np.repeat(np.asarray(d, np.float64), BLOCK8)[:k.size]
    return rn32(rn32(k * np.abs(k)) * step)


def adamw_moments(g, coef, m, v, beta1: float, beta2: float):
    """(m', v', sqrt(v')) with every operation rounded to float32; coef None leaves g alone."""
    g = np.asarray(g, np.float64)
    if coef is not None:
        g = rn32(g * np.float64(np.float32(coef)))
    b1, w1, b2, w2 = (np.float64(np.float32(t)) for t in (beta1, 1.0 - beta1, beta2, 1.0 - beta2))
    m = rn32(rn32(b1 * np.asarray(m, np.float64)) + rn32(w1 * g))
    v = rn32(rn32(b2 * np.asarray(v, np.float64)) + rn32(w2 * rn32(g * g)))
    return m, v, rn32(np.sqrt(v))


def adamw_param(p, m, v, t: int, lr: float, decay: float, beta1: float, beta2: float, eps: float):
    """(p', the update u) in float64: p' = p - lr (decay p + u), u = m^ / (sqrt(v^) + eps)."""
    p, m, v = (np.asarray(x, np.float64) for x in (p, m, v))
    u = (m / (1.0 - beta1 ** t)) / (np.sqrt(v) / math.sqrt(1.0 - beta2 ** t) + eps)
    return p - lr * (decay * p + u), u


def grad_norm(grads, max_norm: float):
    """(2-norm of all gradients, min(1, max_norm / (norm + 1e-6)))."""
    n = math.sqrt(math.fsum(float(np.square(np.asarray(g, np.float64)).sum()) for g in grads))
    return n, min(1.0, max_norm / (n + 1e-6))


def embed_rows(table_f32, ids, scale: float):
    """RN(scale * table[id]) per token (as float32); ids outside the table give a zero row."""
    w = np.asarray(table_f32, np.float64)
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < w.shape[0])
    y = rn32(w[np.where(ok, ids, 0)] * np.float64(np.float32(scale)))
    y[~ok] = 0.0
    return y.astype(np.float32)


def embed_grad(ids, dy, V: int, scale: float, padding_id: int = -1):
    """(dE, sum of |scale dY| per row, tokens per row) in float64."""
    ids, dy = np.asarray(ids, np.int64), np.asarray(dy, np.float64)
    ok = (ids >= 0) & (ids < V) & (ids != padding_id)
    dE, mag, cnt = np.zeros((V, dy.shape[1])), np.zeros((V, dy.shape[1])), np.zeros(V, np.int64)
    s = np.float64(np.float32(scale))
    np.add.at(dE, ids[ok], s * dy[ok])
    np.add.at(mag, ids[ok], np.abs(s * dy[ok]))
    np.add.at(cnt, ids[ok], 1)
    return dE, mag, cnt
