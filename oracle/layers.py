"""Layer operators in float64 from their definitions (oracle side).

TEST INFRASTRUCTURE (see the package docstring).

Packed layers with bias, activation, gate and residual and their gradient, a
whole layer of experts, and distillation from a teacher's top logits. Written
segment by segment, slot by slot and row by row; nothing is blocked, split or
reordered.
"""
import math

import numpy as np
from scipy.special import erfc

from oracle.dequant import dequantize


def act(name, z):
    """The activation and its slope (at 0, relu's slope is 0)."""
    z = np.asarray(z, np.float64)
    if name == "none":
        return z.copy(), np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if name == "gelu":
        cdf = 0.5 * erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        a, b = math.sqrt(2.0 / math.pi), 0.044715
        t = np.tanh(a * (z + b * z ** 3))
        return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * b * z * z)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def end(z, name, gated):
    """act(z), or act(gate) * other of the two halves of z's columns."""
    d = z.shape[-1] // 2 if gated else z.shape[-1]
    a = act(name, z[..., :d])[0]
    return a * z[..., d:] if gated else a


def linear(X, offsets, qweight, scales, zeros, bits, group, name, gated, before, before_z, bias=None, residual=None,
           rows=None):
    """(Y, Z) over the segments; other rows as in `before` and `before_z`."""
    Y, Z = np.array(before, np.float64), np.array(before_z, np.float64)
    n = X.shape[1]
    for e in range(len(offsets) - 1):
        W = dequantize(qweight[e], scales[e], zeros[e], bits, group, n)
        for p in range(offsets[e], offsets[e + 1]):
            Z[p] = np.asarray(X[p if rows is None else rows[p]], np.float64) @ W.T
            if bias is not None:
                Z[p] += np.asarray(bias[e], np.float64)
            Y[p] = end(Z[p], name, gated)
            if residual is not None:
                Y[p] += np.asarray(residual[p], np.float64)
    return Y, Z


def linear_grad(dY, Z, offsets, qweight, scales, zeros, bits, group, n, name, gated, before_z, before):
    """(dX, dZ, dbias); rows outside the segments as in `before` and `before_z`."""
    dZ, dX = np.array(before_z, np.float64), np.array(before, np.float64)
    d = dY.shape[1]
    db = np.zeros((len(offsets) - 1, dZ.shape[1]))
    for e in range(len(offsets) - 1):
        W = dequantize(qweight[e], scales[e], zeros[e], bits, group, n)
        for p in range(offsets[e], offsets[e + 1]):
            g = np.asarray(dY[p], np.float64)
            z = None if Z is None else np.asarray(Z[p], np.float64)
            if gated:
                a, slope = act(name, z[:d])
                dZ[p] = np.concatenate([g * z[d:] * slope, g * a])
            else:
                dZ[p] = g if z is None else g * act(name, z)[1]
            db[e] += dZ[p]
            dX[p] = dZ[p] @ W
    return dX, dZ, db


def expert_layer(X, ids, weights, up, down, bits, group, name, gated, up_bias=None, down_bias=None, residual=None):
    """Y[t] = residual[t] + sum over the slots j with an expert e of
    weights[t, j] (D_e h + down_bias[e]), h = end(U_e x_t + up_bias[e])."""
    T, n = X.shape
    E = up[0].shape[0]
    d = up[0].shape[1] // (2 if gated else 1)
    Y = np.zeros((T, n)) if residual is None else np.array(residual, np.float64)
    for e in range(E):
        if not np.any(ids == e):
            continue
        U = dequantize(up[0][e], up[1][e], up[2][e], bits, group, n)
        D = dequantize(down[0][e], down[1][e], down[2][e], bits, group, d)
        for t in range(T):
            for j in range(ids.shape[1]):
                if ids[t, j] != e:
                    continue
                z = U @ np.asarray(X[t], np.float64)
                if up_bias is not None:
                    z = z + np.asarray(up_bias[e], np.float64)
                o = D @ end(z, name, gated)
                if down_bias is not None:
                    o = o + np.asarray(down_bias[e], np.float64)
                Y[t] += float(weights[t, j]) * o
    return Y


def distill(Z, ids, teacher, temperature, log_probs):
    """(loss, lse, p): p lists each row's (id, probability) pairs."""
    T, V = Z.shape
    loss, lse, ps = np.zeros(T), np.zeros(T), []
    for t in range(T):
        s = np.asarray(Z[t], np.float64) / temperature
        top = s.max()
        lse[t] = top + math.log(np.exp(s - top).sum()) if math.isfinite(top) else top
        at = [k for k in range(ids.shape[1]) if 0 <= ids[t, k] < V]
        x = np.array([float(teacher[t, k]) for k in at])
        if log_probs:
            p = np.exp(x)
        elif len(at) and x.max() > -np.inf:
            p = np.exp((x - x.max()) / temperature)
            p /= p.sum()
        else:
            p = np.zeros(len(at))
        ps.append([(int(ids[t, k]), float(v)) for k, v in zip(at, p)])
        for v, pk in ps[-1]:
            if pk > 0:
                loss[t] += pk * (math.log(pk) - (s[v] - lse[t]))
    return loss, lse, ps


def distill_grad(Z, lse, ps, grad, temperature):
    T, V = Z.shape
    dZ = np.zeros((T, V))
    for t in range(T):
        mass = sum(p for _, p in ps[t])
        if mass == 0:
            continue
        dZ[t] = mass * np.exp(np.asarray(Z[t], np.float64) / temperature - lse[t])
        for v, p in ps[t]:
            dZ[t, v] -= p
        dZ[t] *= float(grad[t]) / temperature
    return dZ
