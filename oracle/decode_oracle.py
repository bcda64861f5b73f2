"""Plain fp64 numpy forms of the 8-bit head and of sampling: rows quantised to
int8, the product of int8 rows, and one draw per row of logits (the formulas
of include/fkl.h, fkl_quantize / fkl_project / fkl_sample)."""

from __future__ import annotations

import numpy as np


def quantize(x):
    """(levels int8 [M, K], scale fp32 [M]) of the rows of x (any float type).

    127 x is exact in fp64 for x of up to 24 significant bits, and the fp64
    quotient of two such numbers is a half exactly when the real one is, and
    otherwise on the same side of it."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x).max(axis=1)
    bad = ~np.isfinite(a)
    safe = np.where(bad | (a == 0), 1.0, a)
    q = np.rint(np.where(bad[:, None], 0.0, x) * 127.0 / safe[:, None])
    scale = (np.where(bad, np.nan, a).astype(np.float32) / np.float32(127.0)).astype(np.float32)
    return q.astype(np.int8), scale


def project(a, a_scale, b, b_scale, bias=None):
    """(result fp64 [M, N], its part before the bias)."""
    s = np.asarray(a).astype(np.int64) @ np.asarray(b).astype(np.int64).T
    prod = s * np.asarray(a_scale, np.float64)[:, None] * np.asarray(b_scale, np.float64)[None, :]
    return (prod if bias is None else prod + np.asarray(bias, np.float64)[None, :]), prod


def kept_entries(x, T, k, p, q):
    """(kept positions ascending, their weights) of one row; empty if every entry is masked."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    V = x.size
    if not (np.isfinite(T) and T >= 0) or not (x > -np.inf).any():
        return np.empty(0, np.int64), np.empty(0)
    order = np.lexsort((np.arange(V), -x))
    m = x[order[0]]
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        w = np.exp((x - m) / T) if T > 0 else np.zeros(V)
    w[x == -np.inf] = 0.0
    w[x == m] = 1.0
    first = T == 0 or p <= 0 or q > 1
    n = 1 if first else V if k <= 0 or k > V else k
    order = order[:n]
    ws = w[order]
    before = np.concatenate([[0.0], np.cumsum(ws)[:-1]])
    keep = np.ones(n, bool)
    if not first and p < 1:
        keep &= before < p * ws.sum()
    if not first and q > 0:
        keep &= ws >= q
    keep[0] = True
    pos = np.sort(order[keep])
    return pos, w[pos]


def sample(logits, u, T=1.0, k=0, p=1.0, q=0.0, ids=None):
    """(token int32 [N], logprob fp64 [N]); T, k, p, q numbers or arrays [N].
    The fp32 settings are taken as fp32 values."""
    logits = np.asarray(logits, dtype=np.float64)
    N, V = logits.shape
    T, p, q = (np.broadcast_to(np.asarray(v, np.float32), (N,)).astype(np.float64) for v in (T, p, q))
    p, q = np.where(np.isnan(p), 1.0, p), np.where(np.isnan(q), 0.0, q)
    k = np.broadcast_to(np.asarray(k, np.int64), (N,))
    token, logprob = np.full(N, -1, np.int32), np.full(N, -np.inf)
    for r in range(N):
        pos, w = kept_entries(logits[r], T[r], k[r], p[r], q[r])
        if pos.size == 0:
            continue
        ur = float(u[r])
        ur = 0.0 if not ur > 0 else min(ur, 1.0)
        run = np.cumsum(w)
        hit = np.flatnonzero(run > ur * run[-1])
        i = hit[0] if hit.size else np.flatnonzero(w > 0)[-1]
        token[r] = pos[i] if ids is None else ids[r, pos[i]]
        logprob[r] = np.log(w[i] / run[-1])
    return token, logprob
