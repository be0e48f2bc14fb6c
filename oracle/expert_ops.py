"""Float64 oracle of the expert layer's separate operators: plain numpy loops over
the definitions (rows by expert and back, their gradients, the gradient of the
routing softmax, rows times 4-bit weights and the gradient to the rows).

Test infrastructure only; nothing here is shared with the product path.  Arrays
come in as float64 (decoded by the caller) or integers, results are float64.
"""

from __future__ import annotations

import numpy as np

from oracle import mxfp4_moe as O


def permute(x, sorted_pairs, top_k):
    """(rows, pair_rows): empty rows are zeros, a pair listed twice belongs to its later row."""
    T, H = x.shape
    rows = np.zeros((len(sorted_pairs), H))
    pair_rows = np.full(T * top_k, -1, dtype=np.int64)
    for i, p in enumerate(sorted_pairs):
        if 0 <= p < T * top_k:
            rows[i] = x[p // top_k]
            pair_rows[p] = i
    return rows, pair_rows


def unpermute(rows, pair_rows, weights):
    """(y, sum of the terms' magnitudes): the second bounds the rounding of the fp32 sum."""
    T, k = weights.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for p, r in enumerate(pair_rows):
        if 0 <= r < len(rows):
            t, j = divmod(p, k)
            y[t] += weights[t, j] * rows[r]
            mag[t] += abs(weights[t, j]) * np.abs(rows[r])
    return y, mag


def unpermute_backward(dy, rows, sorted_pairs, pair_rows, weights):
    """(d_rows, d_weights, sum of the dot products' magnitudes)."""
    T, k = weights.shape
    d_rows, d_w, mag = np.zeros_like(rows), np.zeros((T, k)), np.zeros((T, k))
    for p, r in enumerate(pair_rows):
        if 0 <= r < len(rows):
            t, j = divmod(p, k)
            d_w[t, j] = np.dot(dy[t], rows[r])
            mag[t, j] = np.dot(np.abs(dy[t]), np.abs(rows[r]))
            if sorted_pairs[r] == p:
                d_rows[r] = weights[t, j] * dy[t]
    return d_rows, d_w, mag


def route_backward(ids, weights, d_weights, num_experts):
    out = np.zeros((len(ids), num_experts))
    for t in range(len(ids)):
        mean = sum(weights[t, j] * d_weights[t, j] for j in range(ids.shape[1]))
        for j, e in enumerate(ids[t]):
            if 0 <= e < num_experts:
                out[t, e] += weights[t, j] * (d_weights[t, j] - mean)
    return out


def weights_of(blocks, scales, scale2=None):
    """Float64 weights [..., N, K] of codes [..., N, K/2] with E8M0 scales per 32, or, with
    scale2 (a number or [E]), E4M3 scales per 16 and the second-level scale."""
    if scale2 is None:
        return O.dequantize_f64(blocks, scales)
    s2 = np.asarray(scale2, dtype=np.float64)
    return O.nvfp4_dequantize_f64(blocks, scales) * (s2.reshape(-1, 1, 1) if blocks.ndim == 3 else s2.reshape(()))


def linear(x, w, offsets=None, bias=None):
    """(y, sum of the products' magnitudes, rows written): x [R, K], w [E, N, K] (or [N, K])."""
    if w.ndim == 2:
        w, offsets = w[None], [0, len(x)]
        bias = None if bias is None else bias[None]
    R, N = len(x), w.shape[1]
    y, mag, written = np.zeros((R, N)), np.zeros((R, N)), np.zeros(R, dtype=bool)
    for e in range(len(w)):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
        if bias is not None:
            y[a:b] += bias[e]
            mag[a:b] += np.abs(bias[e])
        written[a:b] = True
    return y, mag, written


def linear_backward(dy, w, offsets=None):
    """(dx, sum of the products' magnitudes, rows written): dy [R, N], w [E, N, K] (or [N, K])."""
    return linear(dy, np.swapaxes(w, -1, -2), offsets)
