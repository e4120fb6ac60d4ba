"""Expert operators in float64 from their definitions (oracle side).

TEST INFRASTRUCTURE (see the package docstring).

Rows in the order of their experts, the way there and back, the packed
products of several layers over segments of rows, and activations kept in 8
bits. Everything is written slot by slot or segment by segment; nothing is
sorted, blocked or factored.
"""
import math

import numpy as np

from oracle.dequant import dequantize


def route(ids, E):
    """(offsets, rows, inverse): every kept slot takes the next free place of
    its expert, in slot order."""
    ids = np.asarray(ids)
    T, k = ids.shape
    counts = [0] * E
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                counts[ids[t, j]] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    free = list(offsets[:-1])
    rows = np.full(T * k, -1, np.int32)
    inverse = np.full((T, k), -1, np.int32)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                inverse[t, j] = free[e]
                rows[free[e]] = t
                free[e] += 1
    return np.array(offsets, np.int32), rows, inverse


def dispatch(X, inverse, before):
    """Rows of X at their places; the others as in `before`."""
    out = np.array(before)
    T, k = inverse.shape
    for t in range(T):
        for j in range(k):
            if 0 <= inverse[t, j] < out.shape[0]:
                out[inverse[t, j]] = X[t]
    return out


def combine(Ys, inverse, weights=None):
    T, k = inverse.shape
    Y = np.zeros((T, Ys.shape[1]))
    for t in range(T):
        for j in range(k):
            p = inverse[t, j]
            if 0 <= p < Ys.shape[0]:
                Y[t] += (1.0 if weights is None else float(weights[t, j])) * np.asarray(Ys[p], np.float64)
    return Y


def combine_grad(dY, Ys, inverse, weights, before):
    dYs = np.array(before, np.float64)
    T, k = inverse.shape
    dw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = inverse[t, j]
            if 0 <= p < Ys.shape[0]:
                dYs[p] = float(weights[t, j]) * np.asarray(dY[t], np.float64)
                dw[t, j] = np.asarray(dY[t], np.float64) @ np.asarray(Ys[p], np.float64)
    return dYs, dw


def expert_matmul(X, offsets, qweight, scales, zeros, bits, group, n, rows=None, before=None):
    """Y[p] = X[rows[p]] W_hat_e^T over the segments; other rows as in `before`."""
    out = np.array(before, np.float64)
    for e in range(len(offsets) - 1):
        W = dequantize(qweight[e], scales[e], zeros[e], bits, group, n)
        for p in range(offsets[e], offsets[e + 1]):
            out[p] = np.asarray(X[p if rows is None else rows[p]], np.float64) @ W.T
    return out


def expert_matmul_grad(dY, offsets, qweight, scales, zeros, bits, group, n, before):
    out = np.array(before, np.float64)
    for e in range(len(offsets) - 1):
        W = dequantize(qweight[e], scales[e], zeros[e], bits, group, n)
        lo, hi = offsets[e], offsets[e + 1]
        out[lo:hi] = np.asarray(dY[lo:hi], np.float64) @ W
    return out


def keep(X):
    """(codes, exps, values) of the 8-bit copy, group by group: 2^p <= max|x|
    < 2^(p + 1), p at least -120, step 2^(p - 6)."""
    X = np.asarray(X, np.float64)
    T, n = X.shape
    groups = (n + 31) // 32
    codes = np.zeros((T, 32 * groups), np.int8)
    exps = np.zeros((T, groups), np.uint8)
    values = np.zeros((T, n))
    for t in range(T):
        for g in range(groups):
            x = X[t, 32 * g:32 * g + 32]
            if not np.all(np.isfinite(x)):
                exps[t, g] = 255
                values[t, 32 * g:32 * g + 32] = np.nan
                continue
            top = float(np.abs(x).max())
            p = max(math.frexp(top)[1] - 1, -120) if top > 0 else -120
            step = math.ldexp(1.0, p - 6)
            exps[t, g] = p - 6 + 127
            for i, v in enumerate(x):
                c = max(-127, min(127, round(v / step)))      # half to even
                codes[t, 32 * g + i] = c
                values[t, 32 * g + i] = c * step
    return codes, exps, values


def weight_grad(P, values, offsets, rows=None):
    """G[e] = sum over the rows p of segment e of P[p]^T values[rows[p]]."""
    E = len(offsets) - 1
    G = np.zeros((E, P.shape[1], values.shape[1]))
    for e in range(E):
        for p in range(offsets[e], offsets[e + 1]):
            G[e] += np.outer(np.asarray(P[p], np.float64), values[p if rows is None else rows[p]])
    return G
