"""Oracle of the operators of a block around the packed linears: the product's
epilogue and its backward pass, the gradient of the product's input, layer and
RMS norm with their backward pass, and a router's balance loss, in float64 from
their definitions (include/awq.h states them)."""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erf

from .awq import unpack_codes


def dequantized(words, step, zeros, group):
    """[N, K/8] packed words -> [N, K] weights."""
    q = unpack_codes(words).astype(np.float64)
    return (q - np.repeat(zeros.astype(np.float64), group, axis=1)) * np.repeat(step.astype(np.float64), group, axis=1)


def _sigma(z):
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


_C = math.sqrt(2.0 / math.pi)


def act_value(act, z):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + erf(z / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * _sigma(z)
    return z


def act_slope(act, z):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * (1.0 + erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        return _sigma(z) * (1.0 + z * _sigma(-z))
    return np.ones_like(z)


def layer_norm(x, weight, bias, eps, rms):
    """(y, mean, rstd)."""
    mean = np.zeros(x.shape[0]) if rms else x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None] * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, rms):
    """(dx, dweight, dbias)."""
    xh = (x if rms else x - mean[:, None]) * rstd[:, None]
    a = dy * weight
    inner = a - xh * (a * xh).mean(axis=1, keepdims=True)
    if not rms:
        inner = inner - a.mean(axis=1, keepdims=True)
    return inner * rstd[:, None], (dy * xh).sum(axis=0), dy.sum(axis=0)


def balance_loss(logits, ids, coef, sigmoid=False, mask=None, grad=1.0):
    """(loss, counts, slope, dlogits)."""
    T, E = logits.shape
    p = np.zeros((T, E))
    rest = np.ones((T, E))
    counts = np.zeros(E, np.int64)
    rows = 0
    for t in range(T):
        row = logits[t].astype(np.float64)
        usable = ~np.isnan(row) & (row > -np.inf)
        if (mask is not None and not mask[t]) or not usable.any():
            continue
        rows += 1
        l = np.minimum(row[usable], float(np.finfo(np.float32).max))
        if sigmoid:
            # log sigma keeps what a sigma of very low logits would lose
            s = np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))
            rest[t, usable] = _sigma(-l)
        else:
            s = l
        s = np.exp(s - s.max())
        p[t, usable] = s / s.sum()
        for i in ids[t]:
            if 0 <= i < E:
                counts[i] += 1
    n = counts.sum()
    slope = coef * E * counts / (n * rows) if n and rows else np.zeros(E)
    dl = grad * p * (slope - (p * slope).sum(axis=1, keepdims=True))
    return float((slope * p.sum(axis=0)).sum()), counts, slope, dl * rest if sigmoid else dl
