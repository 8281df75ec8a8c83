"""Float64 oracle of the operators for unquantised experts: products with bias,
activation and residual, the gradient through them, clipping by the global norm,
and the layer on 16-bit experts; and the error bounds the GPU tests use.
"""

from __future__ import annotations

import numpy as np
from scipy.special import erfc

from . import linear as ol

U = 2.0 ** -24   # half a step of f32
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
C = np.sqrt(2.0 / np.pi)
A = 0.044715


def sigmoid(z):
    z = np.asarray(z, np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _inner(z):
    """t of gelu_tanh = z sigmoid(t)."""
    return 2.0 * C * (z + A * z ** 3)


def act(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * sigmoid(z)
    if name == "gelu":
        return 0.5 * z * erfc(-z / np.sqrt(2.0))
    if name == "gelu_tanh":
        return z * sigmoid(_inner(z))
    return z


def slope(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = sigmoid(z)
        return s + z * s * sigmoid(-z)
    if name == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        t = _inner(z)
        return sigmoid(t) + z * sigmoid(t) * sigmoid(-t) * 2.0 * C * (1.0 + 3.0 * A * z * z)
    return np.ones_like(z)


MAX_SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}


def act_rel(name, z):
    """Relative error of act(z) * u in f32 from an exact z: a dozen operations of
    one rounding or one ulp each (2 U), and the rounding of the exponent, which
    counts by its size: z^2 / 2 of the gelus' tails, twice over for its parts."""
    z = np.asarray(z, np.float64)
    if name in ("none", "relu"):
        return np.full(z.shape, U)
    if name == "silu":
        return np.full(z.shape, 24 * U)
    if name == "gelu":
        return (24 + 4 * z * z) * U
    return (24 + 4 * np.abs(_inner(z))) * U


def slope_tol(name, z):
    """|act'(z) in f32 - act'(z)|: the same of each of its terms, whose magnitudes
    are summed."""
    z = np.asarray(z, np.float64)
    if name in ("none", "relu"):
        return np.zeros(z.shape)
    if name == "silu":
        return 32 * U * (sigmoid(z) + np.abs(z) * sigmoid(z) * sigmoid(-z))
    if name == "gelu":
        m = 0.5 * erfc(-z / np.sqrt(2.0)) + np.abs(z) * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
        return (32 + 4 * z * z) * U * m
    t = _inner(z)
    m = sigmoid(t) + np.abs(z) * sigmoid(t) * sigmoid(-t) * 2.0 * C * (1.0 + 3.0 * A * z * z)
    return (32 + 4 * np.abs(t)) * U * m


def linear_act(x, w, bias=None, residual=None, name="none", gated=False, offsets=None):
    """(y, its bound before the output's rounding, z, its bound)."""
    z, tz = ol.grouped(x, w, offsets)
    for g, (lo, hi) in enumerate(ol.spans(offsets, x.shape[0])):
        if bias is not None:
            z[lo:hi] += bias[g]
    tz = tz + U * np.abs(z)
    if gated:
        F = w.shape[1] // 2
        (a, u), (ta, tu) = np.split(z, [F], 1), np.split(tz, [F], 1)
        f = act(name, a)
        y = f * u
        t = (MAX_SLOPE[name] * ta) * (np.abs(u) + tu) + np.abs(f) * tu + act_rel(name, a) * np.abs(y) + U * np.abs(y)
    else:
        y = act(name, z)
        t = MAX_SLOPE[name] * tz + act_rel(name, z) * np.abs(y)
    if residual is not None:
        y = y + residual
        t = t + U * np.abs(y)
    return y, t, z, tz


def act_backward(dy, z, groups, name="none", gated=False, offsets=None):
    """(dz, its bound before the output's rounding, db, its bound)."""
    if gated:
        a, u = np.split(z, [z.shape[1] // 2], 1)
        f, s = act(name, a), slope(name, a)
        dz = np.concatenate([dy * u * s, dy * f], 1)
        t = np.concatenate([np.abs(dy * u) * slope_tol(name, a), np.abs(dy * f) * act_rel(name, a)], 1)
    else:
        dz = dy * slope(name, z)
        t = np.abs(dy) * slope_tol(name, z)
    t = t + 2 * U * np.abs(dz)
    db, tb = np.zeros((groups, z.shape[1])), np.zeros((groups, z.shape[1]))
    for g, (lo, hi) in enumerate(ol.spans(offsets, z.shape[0])):
        db[g] = dz[lo:hi].sum(0)
        # f32 additions one after the other: a thread's rows, a block's row classes, its partial sums
        depth = min(hi - lo, 64 + 256 + (hi - lo) // 64 + 16)
        tb[g] = t[lo:hi].sum(0) + depth * U * (np.abs(dz[lo:hi]) + t[lo:hi]).sum(0)
    return dz, t, db, tb


def clip(grads, max_norm):
    """(norm, factor) in float64."""
    norm = float(np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads)))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def layer(x, w1, w2, phys, topk_w, p0, eps):
    """The layer on the pairs (t, j) of phys / topk_w [T, k]: (out, its bound
    before the output's rounding).  w * act is held in f32 and enters the second
    product in three parts, which lose nothing above f32's smallest normal number, in f16
    (eps 2^-10) nothing above 2^-38 of the largest of 64 columns; sums of three products a
    column, and of one value every 64 columns.  topk_w: float64 weights, 4e-6 of their
    value uncertain."""
    T, H = x.shape
    F = w2.shape[2]
    out, tol, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    pairs = 0
    for t in range(T):
        for j in range(phys.shape[1]):
            s = int(phys[t, j]) - p0
            if not 0 <= s < w1.shape[0]:
                continue
            pairs = max(pairs, j + 1)
            h = w1[s] @ x[t]
            th = ol.sum_bound(H) * (np.abs(w1[s]) @ np.abs(x[t]))
            a, u = h[:F], h[F:]
            f, w = act("silu", a), topk_w[t, j]
            v = f * u * w
            tv = w * (1.1 * th[:F] * (np.abs(u) + th[F:]) + np.abs(f) * th[F:]) + (24 * U + 4e-6) * np.abs(v)
            tv += 2.0 ** -126
            if eps == 2.0 ** -10:
                top = np.maximum.reduceat(np.abs(v) + tv, np.arange(0, F, 64))
                tv += 2.0 ** -38 * np.repeat(top, 64)[:F]
            out[t] += w2[s] @ v
            tol[t] += np.abs(w2[s]) @ tv
            mag[t] += np.abs(w2[s]) @ (np.abs(v) + tv)
    n = F * max(pairs, 1)
    return out, tol + ol.sum_bound(3 * n + n // 8) * mag   # (four roundings for 32 products: n / 64 sums are as 8 n / 64)
