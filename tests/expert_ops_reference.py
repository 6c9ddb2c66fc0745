"""The FP8 expert operators in 64 bits, written from their definitions."""

import numpy as np
import torch

FLOOR = 2.0 ** -96


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def route(logits, top_k, bias=None, softmax=False, n_groups=1, top_groups=1, top2=False, renorm=True, scale=1.0):
    """ids, w of logits [T][E] (float64).  Keys are the logits, or score + bias."""
    T, E = logits.shape
    ids, w = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    size = E // n_groups
    for t in range(T):
        x = logits[t]
        open_ = x > -np.inf
        score = np.zeros(E)
        with np.errstate(over="ignore"):
            if softmax:
                if open_.any():
                    m = x[open_].max()
                    u = np.where(open_, np.exp(np.where(x == m, 0.0, np.where(open_, x, 0.0) - (m if np.isfinite(m) else np.inf))), 0.0)
                    score = u / u.sum()
            else:
                score[open_] = 1 / (1 + np.exp(-x[open_]))
        key = np.where(open_, x if bias is None else score + bias, -np.inf)
        key = np.where(key > -np.inf, key, -np.inf)
        if n_groups > 1:
            gs = np.full(n_groups, -np.inf)
            for g in range(n_groups):
                part = slice(g * size, (g + 1) * size)
                v = (score if top2 and bias is None else key)[part][key[part] > -np.inf]
                if v.size:
                    gs[g] = np.sort(v)[-2:].sum() if top2 else v.max()
            for g in np.argsort(-gs, kind="stable")[top_groups:]:
                key[g * size:(g + 1) * size] = -np.inf
        best = np.argsort(-key, kind="stable")[:top_k]
        best = best[key[best] > -np.inf]
        if best.size == 0:
            continue
        ids[t, :best.size] = best
        s = score[best]
        if renorm:
            xs = x[best]
            if softmax:
                m = xs.max()
                u = np.exp(np.where(xs == m, 0.0, xs - (m if np.isfinite(m) else np.inf)))
            else:  # scores times one factor, which keeps very low ones apart from zero
                low = np.minimum(xs, 0)
                u = np.exp(np.where(low == low.max(), 0.0, low - low.max())) / (1 + np.exp(-np.abs(xs)))
            s = u / u.sum()
        w[t, :best.size] = scale * s
    return ids, w


def group(ids, E):
    ids = np.asarray(ids).reshape(-1)
    ok = (ids >= 0) & (ids < E)
    order_ok = np.argsort(np.where(ok, ids, E), kind="stable")[:ok.sum()]
    order, pos = np.full(ids.size, -1, np.int32), np.full(ids.size, -1, np.int32)
    order[:ok.sum()] = order_ok
    pos[order_ok] = np.arange(ok.sum())
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[ok], minlength=E))]).astype(np.int32)
    return offsets, order, pos


def quantise_values(x):
    """(codes' values, scales [kb][rows], quotients) of x [rows][K] in 64 bits."""
    rows, K = x.shape
    kb = -(-K // 128)
    q, scales = np.empty_like(x), np.empty((kb, rows))
    v = np.empty_like(x)
    for b in range(kb):
        p = slice(b * 128, min(K, (b + 1) * 128))
        s = np.maximum(np.abs(x[:, p]).max(1), FLOOR) / 448
        scales[b] = s
        v[:, p] = x[:, p] / s[:, None]
        unit = e4m3_step(v[:, p])
        q[:, p] = np.rint(v[:, p] / unit) * unit
    return q, scales, v


def e4m3_step(v):
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)


def expand_scales(s, K):
    return np.repeat(s, 128, axis=0)[:K]


def gemm(a, sa, b, sb, offsets=None):
    """y and the sum of the magnitudes of its terms, both [M][N] (rows of no expert: NaN)."""
    M, K = a.shape
    E, N, _ = b.shape
    y, mag = np.full((M, N), np.nan), np.full((M, N), np.nan)
    edge = [0, M] if offsets is None else list(offsets)
    A = a * expand_scales(sa, K).T
    for e in range(E):
        lo, hi = int(edge[e]), int(edge[e + 1])
        if hi <= lo:
            continue
        B = b[e] * np.repeat(np.repeat(sb[e], 128, axis=0)[:N], 128, axis=1)[:, :K]
        y[lo:hi] = A[lo:hi] @ B.T
        mag[lo:hi] = np.abs(A[lo:hi]) @ np.abs(B).T
    return y, mag


def combine(rows, pos, w, shared=None):
    T, k = pos.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for j in range(k):
        on = (pos[:, j] >= 0) & (pos[:, j] < rows.shape[0])
        term = w[on, j][:, None] * rows[pos[on, j]]
        y[on] += term
        mag[on] += np.abs(term)
    if shared is not None:
        y += shared
        mag += np.abs(shared)
    return y, mag
