"""Definitions of the operators of a step with trees of drafted tokens, in 64 bits.

Plain NumPy, one segment after another; what the CUDA kernels compute is compared with
this.  Attention also returns, per value, the sum that its error bound is made of.
"""

from __future__ import annotations

import numpy as np


def tree_rows(parents):
    """(bits [n, n], depth [n]): which tokens each token of one tree sees.  A parent that is
    not before its token counts as none."""
    n = len(parents)
    bits = np.zeros((n, n), dtype=bool)
    depth = np.zeros(n, dtype=np.int64)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            bits[i] = bits[p]
            depth[i] = depth[p] + 1
        bits[i, i] = True
    return bits, depth


def pack(bits, words):
    """[n, <= 32 words] truth values to int32 words, bit 0 of word 0 the first."""
    n, k = bits.shape
    full = np.zeros((n, 32 * words), dtype=np.uint32)
    full[:, :k] = bits
    w = (full.reshape(n, words, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint64)
    return w.astype(np.uint32).view(np.int32)


def tree_attention(q, k, v, hist, bits, scale):
    """One segment: q [n, H_q, D], k and v [hist + n, H_kv, D] (float64), bits [n, n] (only
    tokens before a token and itself count).  Returns (out [n, H_q, D], lse [n, H_q], mass
    [n, H_q, D] = softmax times |v|)."""
    n, hq, _ = q.shape
    G = hq // k.shape[1]
    see = np.ones((n, hist + n), dtype=bool)
    see[:, hist:] = (np.tril(bits, -1) | np.eye(n, dtype=bool))
    out, mass = np.empty_like(q), np.empty_like(q)
    lse = np.empty((n, hq))
    for h in range(hq):
        kh, vh = k[:, h // G], v[:, h // G]
        for i in range(n):
            x = (kh[see[i]] @ q[i, h]) * scale
            m = x.max()
            e = np.exp(x - m)
            lse[i, h] = m + np.log(e.sum())
            w = e / e.sum()
            out[i, h] = w @ vh[see[i]]
            mass[i, h] = w @ np.abs(vh[see[i]])
    return out, lse, mass


def _clean(x):
    x = np.asarray(x, dtype=np.float64)
    return np.where((x > 0) & (x < np.inf), x, 0.0)


def _pick(w, u):
    """First place whose prefix sum is above u times the sum; -1 without a positive entry."""
    if not w.sum() > 0:
        return -1
    s = np.cumsum(w)
    at = np.flatnonzero((w > 0) & (s > u * s[-1]))
    return int(at[0]) if len(at) else int(np.flatnonzero(w > 0)[-1])


def verify(target, tokens, u, u_last, parents=None, draft=None):
    """One segment of n rows.  Returns (path, new tokens), as many of each."""
    n, V = target.shape
    cur, c, mass, path, new, gone = 0, 0.0, 1.0, [0], [], set()
    for i in range(1, n):
        up = i - 1 if parents is None else int(parents[i])
        x = int(tokens[i])
        if up != cur or up >= i or not 0 <= x < V:
            continue
        p = float(_clean(target[cur, x]))
        if draft is not None:
            q = float(_clean(draft[cur, x]))
            ok = float(u[i]) * mass * q < p - c * q
        else:
            ok = x not in gone and float(u[i]) * mass < p
        if ok:
            path.append(i)
            new.append(x)
            cur, c, mass, gone = i, 0.0, 1.0, set()
        elif draft is not None:
            c += mass
            mass = np.maximum(_clean(target[cur]) - c * _clean(draft[cur]), 0).sum()
        elif x not in gone:
            gone.add(x)
            mass = max(mass - p, 0.0)
    p = _clean(target[cur])
    w = p.copy()
    if draft is not None:
        w = np.maximum(p - c * _clean(draft[cur]), 0)
    elif gone:
        w[list(gone)] = 0
    if not w.sum() > 0:
        w = p
    new.append(_pick(w, float(u_last)))
    return path, new


def keep(cache, table, hist, path, page_size):
    """One segment in one cache [pages, P, ...], in place."""
    rows = [cache[table[(hist + a) // page_size], (hist + a) % page_size].copy() for a in path]
    for k, row in enumerate(rows):
        cache[table[(hist + k) // page_size], (hist + k) % page_size] = row
