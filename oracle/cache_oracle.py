"""Plain numpy float64 forms of the operators of a decoder's paged cache:
norm and rotation of query and key heads, append to page pools, attention of
drafted rows over cache and tree.

Test infrastructure only.  It shares no code with the CUDA path and follows
the definitions in include/specfold.h row by row.
"""
from __future__ import annotations

import numpy as np

PAD = -2


def angles(positions, hd, theta):
    """positions[t] * theta^(-2j/hd) reduced to one turn, in extended precision."""
    j = np.arange(hd // 2, dtype=np.longdouble)
    a = np.asarray(positions, np.longdouble)[:, None] * np.power(np.longdouble(theta), -2 * j / hd)
    return np.fmod(a, 2 * np.longdouble(np.pi) + 2 * np.longdouble(1.2246467991473532e-16)).astype(np.float64)


def norm_rotate(x, gain, eps, positions, theta):
    """x [T, heads, hd] -> (out, size): size bounds |y[j]| + |y[j + hd/2]|, the
    terms that a rotated element sums."""
    y = np.asarray(x, np.float64)
    hd = y.shape[-1]
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    a, b = y[..., :hd // 2], y[..., hd // 2:]
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    if not theta:
        return y, size
    ang = angles(positions, hd, theta)[:, None]
    c, s = np.cos(ang), np.sin(ang)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), size


def slot_of(table, page, num_pages, s, tok):
    """Pool token of sequence s's token, or None."""
    if tok // page >= table.shape[1]:
        return None
    pg = int(table[s, tok // page])
    return pg * page + tok % page if 0 <= pg < num_pages else None


def append(k_pool, v_pool, table, page, K, V, row_start, ctx_len, gk, eps, positions, theta, rows=None):
    """float64 pools after the append; also the pool tokens written and the
    bound of norm_rotate for each."""
    kp, vp = np.asarray(k_pool, np.float64).copy(), np.asarray(v_pool, np.float64).copy()
    num_pages = kp.shape[0] // page
    size = {}
    for s in range(len(ctx_len)):
        for t in range(row_start[s], row_start[s + 1]):
            tok = int(ctx_len[s]) + t - int(row_start[s])
            at = slot_of(table, page, num_pages, s, tok)
            src = t if rows is None else int(rows[t])
            if at is None or not 0 <= src < len(K):
                continue
            pos = tok if positions is None else int(positions[t])
            y, sz = norm_rotate(K[src][None], gk, eps, [pos], theta)
            kp[at], vp[at], size[at] = y[0], V[src], sz[0]
    return kp, vp, size


def ancestors(parent, n):
    """sees[i, j]: row j is row i or one of its ancestors; a padding row sees
    nothing.  parent None: a chain.  Invalid parents count as -1."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        p = i - 1 if parent is None else int(parent[i])
        if p == PAD:
            continue
        sees[i, i] = True
        if 0 <= p < i and (parent is None or parent[p] != PAD):
            sees[i] |= sees[p]
    return sees


def tree_attention(q, k_pool, v_pool, table, page, parent, row_start, ctx_len, scale=None):
    """(o, spread, score): o [T, n_q, hd] (NaN where no sequence owns the row),
    spread = softmax-weighted |v|, score = the largest sum of |q k| * scale."""
    q = np.asarray(q, np.float64)
    T, n_q, hd = q.shape
    n_kv = k_pool.shape[1]
    g = n_q // n_kv
    scale = hd ** -0.5 if not scale else scale
    num_pages = k_pool.shape[0] // page
    o, spread, score = np.full(q.shape, np.nan), np.zeros(q.shape), 0.0
    for s in range(len(ctx_len)):
        a, n, c = int(row_start[s]), int(row_start[s + 1] - row_start[s]), int(ctx_len[s])
        if n == 0:
            continue
        sees = ancestors(None if parent is None else parent[a:a + n], n)
        at = [slot_of(table, page, num_pages, s, t) for t in range(c + n)]
        idx = np.array([0 if x is None else x for x in at])
        k, v = np.asarray(k_pool, np.float64)[idx], np.asarray(v_pool, np.float64)[idx]
        none = np.array([x is None for x in at])
        k[none], v[none] = 0.0, 0.0
        for i in range(n):
            vis = np.concatenate([np.full(c, sees[i].any()), sees[i]])
            if not vis.any():
                o[a + i] = 0.0
                continue
            for h in range(n_q):
                kk, vv = k[vis, h // g], v[vis, h // g]
                w = kk @ q[a + i, h] * scale
                score = max(score, float((np.abs(kk) @ np.abs(q[a + i, h])).max() * scale))
                w = np.exp(w - w.max())
                w /= w.sum()
                o[a + i, h], spread[a + i, h] = w @ vv, w @ np.abs(vv)
    return o, spread, score
