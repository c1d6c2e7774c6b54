"""Oracle of the operators whose weight depends on the row: expert routing, the
routed products and per-row low-rank adapters, in float64 NumPy from their
definitions (include/awq.h states them).  Loops over rows on purpose."""
from __future__ import annotations

import numpy as np

from .awq import unpack_codes


def route_experts(logits, top_k, bias=None, sigmoid=False, n_group=1, topk_group=1, group_top=1, renormalize=True,
                  scale=1.0):
    """(ids [T, top_k] int64, weights [T, top_k] float64)."""
    T, E = logits.shape
    size = E // n_group
    ids = np.full((T, top_k), -1)
    weights = np.zeros((T, top_k))
    for t in range(T):
        row = logits[t].astype(np.float64)
        usable = ~np.isnan(row) & (row > -np.inf)
        row = np.minimum(row, float(np.finfo(np.float32).max))
        score = np.zeros(E)
        if usable.any():
            if sigmoid:
                with np.errstate(over="ignore"):
                    score[usable] = 1.0 / (1.0 + np.exp(-row[usable]))
            else:
                p = np.exp(row[usable] - row[usable].max())
                score[usable] = p / p.sum()
        choice = score + (0.0 if bias is None else bias.astype(np.float64))
        choice[~usable] = -np.inf
        if n_group > 1:
            worth = [np.sort(choice[g * size:(g + 1) * size])[::-1][:group_top].sum() for g in range(n_group)]
            order = sorted(range(n_group), key=lambda g: (-worth[g], g))
            for g in order[topk_group:]:
                choice[g * size:(g + 1) * size] = -np.inf
        order = sorted((e for e in range(E) if choice[e] > -np.inf), key=lambda e: (-choice[e], e))[:top_k]
        ids[t, :len(order)] = order
        w = score[order]
        if renormalize and w.sum() > 0:
            w = w / w.sum()
        weights[t, :len(order)] = w * scale
    return ids, weights


def expert_rows(x, expert, words, step, zero):
    """z[i] = W_{expert[i]} x[i] and, beside it, sum_k |step| (q + z) |x| (the size
    of what a kernel adds up); rows whose expert is outside the stack are 0.
    words [E, N, K/8], step and zero [E, N, G]."""
    E, N, G = step.shape
    K = words.shape[2] * 8
    g = K // G
    out = np.zeros((len(expert), N))
    size = np.zeros((len(expert), N))
    x = x.astype(np.float64)
    for e in np.unique(expert):
        if not 0 <= e < E:
            continue
        rows = np.nonzero(expert == e)[0]
        q = unpack_codes(words[e]).astype(np.float64)
        d = np.repeat(step[e].astype(np.float64), g, axis=1)
        z = np.repeat(zero[e].astype(np.float64), g, axis=1)
        out[rows] = x[rows] @ (d * (q - z)).T
        size[rows] = np.abs(x[rows]) @ (np.abs(d) * (q + z)).T
    return out, size


def swiglu(z):
    n = z.shape[1] // 2
    with np.errstate(over="ignore"):
        return z[:, :n] / (1.0 + np.exp(-z[:, :n])) * z[:, n:]


def lora(x, adapter, a, b, ranks=None, scaling=None):
    """(scaling B A x per row, |scaling| sum |B| |A x|, |scaling| sum |B| |A| |x|)."""
    M, N = x.shape[0], b.shape[1]
    out, size_h, size_x = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    x = x.astype(np.float64)
    for m in range(M):
        i = int(adapter[m])
        if not 0 <= i < a.shape[0]:
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        A, B = a[i, :r].astype(np.float64), b[i, :, :r].astype(np.float64)
        s = 1.0 if scaling is None else float(scaling[i])
        h = A @ x[m]
        out[m] = s * (B @ h)
        size_h[m] = abs(s) * (np.abs(B) @ np.abs(h))
        size_x[m] = abs(s) * (np.abs(B) @ (np.abs(A) @ np.abs(x[m])))
    return out, size_h, size_x
