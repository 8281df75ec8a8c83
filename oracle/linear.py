"""Float64 oracle of the linear operators: fp8 quantisation with a scale per
128 columns, the fp8 product with a scale per block of 128, and the products
grouped by expert with their gradients; and the error bounds the GPU tests use.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
FP8_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quant_scales(x: np.ndarray) -> np.ndarray:
    """f32 scales [rows, ceil(K/128)] of f32 rows: max(amax / 448, 2^-126) in f32."""
    x = np.asarray(x, np.float32)
    s = [np.abs(x[:, c:c + BLOCK]).max(axis=1) / np.float32(FP8_MAX) for c in range(0, x.shape[1], BLOCK)]
    return np.maximum(np.stack(s, axis=1), np.float32(MIN_SCALE))


def spread(s: np.ndarray, n: int, axis: int) -> np.ndarray:
    """Per-block values repeated to n elements along ``axis``."""
    return np.repeat(s, BLOCK, axis=axis).take(range(n), axis=axis)


def swiglu(x: np.ndarray) -> np.ndarray:
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    return g / (1.0 + np.exp(-g)) * u


def spans(offsets, rows: int):
    o = [0, rows] if offsets is None else [int(v) for v in offsets]
    return list(zip(o, o[1:]))


def fp8_linear(xq, xs, w, ws, offsets=None):
    """(y, bound of |GPU sum - y|): the values xq [rows, K] and w [G, N, K] of
    the codes in float64, their scales, and the rows' groups.

    Bound: the matrix instruction takes 32 products at a time (columns
    [16 j, 16 j + 16) and [64 + 16 j, 64 + 16 j + 16) of a block of 128, j < 4),
    aligns them to the largest and may drop what lies 13 binary places below
    its leading bit, so at most 31 of the others lose up to
    2^(floor(log2 largest) - 13) each; the four parts, the scale product, the
    scaled addition and up to 16 partial sums are f32 (2^-24 of the magnitudes
    that occur, three roundings inside a block, three for the scaling)."""
    rows, K = xq.shape
    N = w.shape[1]
    y, tol = np.zeros((rows, N)), np.zeros((rows, N))
    for g, (lo, hi) in enumerate(spans(offsets, rows)):
        mag = np.zeros((hi - lo, N))
        for b in range(blocks(K)):
            c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
            p = xq[lo:hi, None, c] * w[g][None, :, c]
            s = xs[lo:hi, b][:, None] * spread(ws[g][:, b], N, 0)[None, :]
            y[lo:hi] += p.sum(-1) * s
            a = np.abs(np.pad(p, ((0, 0), (0, 0), (0, BLOCK - p.shape[-1]))))
            parts = a.reshape(*a.shape[:2], 2, 4, 16).transpose(0, 1, 3, 2, 4).reshape(*a.shape[:2], 4, 32)
            top = parts.max(-1)
            e = np.floor(np.log2(np.where(top > 0, top, 1.0)))
            drop = np.where(top > 0, 31 * 2.0 ** (e - 13), 0.0).sum(-1)
            tol[lo:hi] += s * (drop + 6 * 2.0 ** -24 * a.sum(-1))
            mag += s * a.sum(-1)
        tol[lo:hi] += (blocks(K) + 16) * 2.0 ** -24 * mag
    return y, tol


def sum_bound(n: int) -> float:
    """|f32 sum of n exact products - exact| over the sum of magnitudes: up to
    four roundings per 32-product instruction and up to 16 partial sums."""
    return (4 * (n / 32 + 1) + 16) * 2.0 ** -24


def grouped(x, w, offsets=None):
    """(y, bound): y[r] = x[r] w[g]^T in float64."""
    rows, N = x.shape[0], w.shape[1]
    y, tol = np.zeros((rows, N)), np.zeros((rows, N))
    for g, (lo, hi) in enumerate(spans(offsets, rows)):
        y[lo:hi] = x[lo:hi] @ w[g].T
        tol[lo:hi] = sum_bound(x.shape[1]) * (np.abs(x[lo:hi]) @ np.abs(w[g]).T)
    return y, tol


def grouped_dx(dy, w, offsets=None):
    return grouped(dy, np.swapaxes(w, 1, 2), offsets)


def grouped_dw(dy, x, groups: int, offsets=None):
    dw, tol = np.zeros((groups, dy.shape[1], x.shape[1])), np.zeros((groups, dy.shape[1], x.shape[1]))
    for g, (lo, hi) in enumerate(spans(offsets, x.shape[0])):
        dw[g] = dy[lo:hi].T @ x[lo:hi]
        tol[g] = sum_bound(hi - lo) * (np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi]))
    return dw, tol
