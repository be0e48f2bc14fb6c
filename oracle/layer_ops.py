"""Float64 oracle of the operators around the expert products: plain numpy over the
definitions (the root-mean-square norm, rows in 8 bits, 8-bit products, the activation,
the balance loss, and their gradients).

Test infrastructure only; nothing here is shared with the product path.  Arrays come in
as float64 (decoded by the caller) or integers, results are float64.  Where a result is
a sum, its terms' magnitudes come beside it, for bounds on the rounding.
"""

from __future__ import annotations

import numpy as np

BLOCK, LARGEST, LEAST = 128, 448.0, 2.0 ** -100


def blocks(n):
    return -(-n // BLOCK)


def e4m3(byte):
    """The value of an E4M3 code (OCP: bias 7, no infinities, S.1111.111 is NaN)."""
    byte = int(byte)
    e, m, sign = (byte >> 3) & 15, byte & 7, -1.0 if byte & 128 else 1.0
    if e == 15 and m == 7:
        return np.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


E4M3 = np.array([e4m3(b) for b in range(256)])


def rms_norm(s, weight, eps):
    """(y, r)"""
    r = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s * r[:, None] * weight, r


def rms_norm_backward(dy, s, weight, eps, d_s=None):
    """(dx, its terms' magnitudes, d_weight, its terms' magnitudes)"""
    r = (1.0 / np.sqrt(np.mean(s * s, axis=1) + eps))[:, None]
    g = dy * weight
    along = np.mean(s * g, axis=1, keepdims=True)
    most = np.mean(np.abs(s * g), axis=1, keepdims=True)
    extra = 0.0 if d_s is None else d_s
    dx = r * g - s * r ** 3 * along + extra
    mag = np.abs(r * g) + np.abs(s) * r ** 3 * most + np.abs(extra)
    return dx, mag, np.sum(dy * s * r, axis=0), np.sum(np.abs(dy * s * r), axis=0)


def block_scales(v):
    """The scale of every block of 128 of the rows."""
    rows, width = v.shape
    out = np.zeros((rows, blocks(width)))
    for j in range(blocks(width)):
        out[:, j] = np.maximum(np.max(np.abs(v[:, BLOCK * j: BLOCK * (j + 1)]), axis=1), LEAST) / LARGEST
    return out


def values(codes, scales):
    """What codes (bytes) and scales of rows stand for."""
    return E4M3[codes] * np.repeat(scales, BLOCK, axis=1)[:, : codes.shape[1]]


def weights(codes, scales):
    """What codes [..., N, K] (bytes) and scales [..., ceil(N/128), ceil(K/128)] stand for."""
    n, k = codes.shape[-2:]
    s = np.repeat(np.repeat(scales, BLOCK, axis=-2)[..., :n, :], BLOCK, axis=-1)[..., :k]
    return E4M3[codes] * s


def swiglu(h, split, alpha, limit, offset):
    gate, up = halves(h, split)
    g, u = np.minimum(gate, limit), np.clip(up, -limit, limit)
    return g * sigmoid(alpha * g) * (u + offset)


def halves(h, split):
    inner = h.shape[1] // 2
    return (h[:, :inner], h[:, inner:]) if split else (h[:, 0::2], h[:, 1::2])


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu_backward(da, h, split, alpha, limit, offset):
    """(dh, the terms' magnitudes)"""
    gate, up = halves(h, split)
    g, u = np.minimum(gate, limit), np.clip(up, -limit, limit)
    s = sigmoid(alpha * g)
    dg = np.where(gate <= limit, da * (u + offset) * s * (1 + alpha * g * (1 - s)), 0.0)
    du = np.where(np.abs(up) <= limit, da * g * s, 0.0)
    mg, mu = np.abs(da * (u + offset)) * s * (1 + np.abs(alpha * g)), np.abs(da * g * s)
    out, mag = np.zeros_like(h), np.zeros_like(h)
    for a, parts in ((out, (dg, du)), (mag, (mg, mu))):
        x, y = halves(a, split)
        x[...], y[...] = parts
    return out, mag


def probabilities(logits):
    """Softmax of each row; zeros for a row without a finite logit."""
    p = np.zeros_like(logits)
    for t, row in enumerate(logits):
        if np.max(row) > -np.inf:
            e = np.exp(row - np.max(row))
            p[t] = e / np.sum(e)
    return p


def balance_loss(logits, ids, mask=None):
    """(loss, counts, density)"""
    T, E = logits.shape
    live = np.ones(T, bool) if mask is None else mask
    counts = np.zeros(E, np.int64)
    for t in np.nonzero(live)[0]:
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
    density = E * counts / max(counts.sum(), 1) / max(int(live.sum()), 1)
    return float(np.sum(probabilities(logits)[live] * density)), counts, density


def balance_loss_backward(logits, density, d_loss, mask=None):
    """(d_logits, the terms' magnitudes)"""
    p = probabilities(logits)
    if mask is not None:
        p = p * mask[:, None]
    mean = np.sum(p * density, axis=1, keepdims=True)
    return d_loss * p * (density - mean), abs(d_loss) * p * (density + mean)
