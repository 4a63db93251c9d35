"""fp64 NumPy definitions of the operators a training step needs beside the
layer: attention with a key window per query row, capped scores and a distance
bias; the per-head norm with the rotary embedding; clipping by the global norm.
Written apart from the layer oracle; its rotation is shared."""
from __future__ import annotations

import numpy as np

from .ref import rope


# ------------------------------------------------------------------ attention

def allowed(s, causal, begin=None, end=None):
    """[s, s] bool: key j is visible to query i iff begin[i] <= j < end[i],
    and j <= i where causal."""
    i, j = np.arange(s)[:, None], np.arange(s)[None]
    ok = np.ones((s, s), bool)
    if causal:
        ok &= j <= i
    if begin is not None:
        ok &= j >= np.asarray(begin)[:, None]
    if end is not None:
        ok &= j < np.asarray(end)[:, None]
    return ok


def attention_mod_head(q, k, v, ok, slope=0.0, cap=0.0, do=None):
    """One head.  q [s, d], k, v [s, d], ok [s, s].  Returns (o, lse), or with
    do (o, lse, dq, dk, dv).  A row that sees nothing has o = 0, lse = -inf and
    gives no gradient."""
    s, d = q.shape
    x = q @ k.T / np.sqrt(d)
    t = np.tanh(x / cap) if cap else None
    y = cap * t if cap else x
    y = y - slope * np.abs(np.arange(s)[:, None] - np.arange(s)[None])
    y = np.where(ok, y, -np.inf)
    some = ok.any(1)
    m = np.where(some, y.max(1, initial=-np.inf), 0.0)
    e = np.where(ok, np.exp(y - m[:, None]), 0.0)
    total = e.sum(1)
    p = e / np.where(some, total, 1.0)[:, None]
    o = p @ v
    with np.errstate(divide="ignore"):
        lse = np.where(some, m + np.log(total), -np.inf)
    if do is None:
        return o, lse
    dp = do @ v.T
    ds = p * (dp - (do * o).sum(1, keepdims=True))
    if cap:
        ds = ds * (1 - t * t)
    ds /= np.sqrt(d)
    return o, lse, ds @ k, ds.T @ q, p.T @ do


def attention_mod(qkv, b, s, H, K, d, causal, begin=None, end=None, slopes=None, cap=0.0, dout=None):
    """The packed layout: qkv [b*s, (H + 2K) d], begin/end [b*s], slopes [H].
    Returns (o [b*s, H d], lse [b, H, s]) or (o, lse, dqkv)."""
    x = np.asarray(qkv, np.float64).reshape(b, s, H + 2 * K, d)
    G = H // K
    o, lse, dx = np.zeros((b, s, H, d)), np.zeros((b, H, s)), np.zeros_like(x)
    do = None if dout is None else np.asarray(dout, np.float64).reshape(b, s, H, d)
    for bi in range(b):
        part = slice(bi * s, (bi + 1) * s)
        ok = allowed(s, causal, None if begin is None else begin[part], None if end is None else end[part])
        for n in range(H):
            g = n // G
            r = attention_mod_head(x[bi, :, n], x[bi, :, H + g], x[bi, :, H + K + g], ok,
                                   0.0 if slopes is None else float(slopes[n]), cap, None if do is None else do[bi, :, n])
            o[bi, :, n], lse[bi, n] = r[0], r[1]
            if do is not None:
                dx[bi, :, n] += r[2]
                dx[bi, :, H + g] += r[3]
                dx[bi, :, H + K + g] += r[4]
    if do is None:
        return o.reshape(b * s, H * d), lse
    return o.reshape(b * s, H * d), lse, dx.reshape(b * s, -1)


# ------------------------------------------------------------------ head norm and rotation

def norm_rope(qkv, s, H, K, d, wq, wk, base, eps, positions=None, dout=None):
    """qkv [rows, (H + 2K) d].  Returns out, or with dout (dqkv, dwq, dwk)."""
    x = np.asarray(qkv, np.float64).reshape(-1, H + 2 * K, d)
    rows = x.shape[0]
    pos = np.arange(rows) % s if positions is None else np.asarray(positions)
    turn = lambda z, inv: rope(z[:, None], base, inverse=inv, positions=pos)[:, 0] if base else z  # noqa: E731
    y = x.copy() if dout is None else np.asarray(dout, np.float64).reshape(x.shape).copy()
    dw = []
    for at, n, w in ((0, H, wq), (H, K, wk)):
        for h in range(at, at + n):
            u = x[:, h]
            r = 1 / np.sqrt((u * u).mean(1, keepdims=True) + eps) if w is not None else np.ones((rows, 1))
            unit = u * r
            if dout is None:
                y[:, h] = turn(unit * w if w is not None else u, False)
                continue
            g = turn(y[:, h], True)
            if w is not None:
                dw.append((g * unit).sum(0))
                g = g * w
                g = r * (g - unit * (g * unit).mean(1, keepdims=True))
            y[:, h] = g
    y = y.reshape(rows, -1)
    if dout is None:
        return y
    return (y, sum(dw[:H]), sum(dw[H:])) if wq is not None else (y, None, None)


# ------------------------------------------------------------------ clipping

def clip(grads, max_norm):
    """(norm, scaled copies)."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(max_norm) else 1.0
    return norm, [np.asarray(g, np.float64) * c for g in grads]
