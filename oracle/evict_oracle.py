"""Plain numpy float64 forms of the rotation by several axes and of the
operators that thin out a paged cache: weights of cached tokens, the choice of
those that stay, and closing the gaps.

Test infrastructure only.  It shares no code with the CUDA path and follows
the definitions in include/specfold.h row by row.
"""
from __future__ import annotations

import numpy as np

from oracle.cache_oracle import slot_of


def axis_pairs(pairs, in_turn):
    """(axis, place among the axis's own pairs) of every rotation pair."""
    if not in_turn:
        return [(a, i) for a, n in enumerate(pairs) for i in range(n)]
    return sorted(((a, i) for a, n in enumerate(pairs) for i in range(n)), key=lambda x: (x[1], x[0]))


def frequencies(pairs, in_turn, theta, own):
    order = axis_pairs(pairs, in_turn)
    half = len(order)
    e = [np.longdouble(i) / pairs[a] if own else np.longdouble(j) / half for j, (a, i) in enumerate(order)]
    return np.power(np.longdouble(theta), -np.array(e, np.longdouble))


def norm_rotate_axes(x, gain, eps, positions, pairs, in_turn, theta, own):
    """x [T, heads, hd], positions [axes, T] -> (out, size), as
    cache_oracle.norm_rotate."""
    y = np.asarray(x, np.float64)
    half = y.shape[-1] // 2
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    a, b = y[..., :half], y[..., half:]
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    axis = [ax for ax, _ in axis_pairs(pairs, in_turn)]
    ang = np.asarray(positions, np.longdouble)[axis].T * frequencies(pairs, in_turn, theta, own)
    ang = np.fmod(ang, 2 * np.longdouble(np.pi) + 2 * np.longdouble(1.2246467991473532e-16)).astype(np.float64)[:, None]
    c, s = np.cos(ang), np.sin(ang)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), size


def weigh(q, k_pool, table, page, row_start, ctx_len, w, decay, rows=None, scale=None):
    """(weights after the call, the share that is new, score = the largest sum
    of |q k| * scale)."""
    q, w = np.asarray(q, np.float64), np.asarray(w, np.float64).copy()
    hd, n_kv = q.shape[2], w.shape[1]
    g = q.shape[1] // n_kv
    scale = hd ** -0.5 if not scale else scale
    num_pages = k_pool.shape[0] // page
    new, score = np.zeros_like(w), 0.0
    for s in range(len(ctx_len)):
        a, n, c = int(row_start[s]), int(row_start[s + 1] - row_start[s]), int(ctx_len[s])
        if n == 0:
            continue
        at = [slot_of(table, page, num_pages, s, t) for t in range(c + n)]
        k = np.asarray(k_pool, np.float64)[[0 if x is None else x for x in at]]
        k[[x is None for x in at]] = 0.0
        for i in range(n):
            r = a + i if rows is None else int(rows[a + i])
            if not 0 <= r < len(q):
                continue
            for h in range(q.shape[1]):
                kk = k[: c + i + 1, h // g]
                x = kk @ q[r, h] * scale
                score = max(score, float((np.abs(kk) @ np.abs(q[r, h])).max() * scale))
                p = np.exp(x - x.max())
                new[s, h // g, : c + i + 1] += p / p.sum()
        old = w[s, :, :c] * decay if decay else 0.0
        w[s, :, :c] = old + new[s, :, :c]
        w[s, :, c:c + n] = new[s, :, c:c + n]
    return w, new, score


def select(weights, lengths, keep, sinks, recent):
    """Per sequence and set the kept tokens, ascending (None: an invalid length)."""
    out = []
    for s, n in enumerate(lengths):
        n = int(n)
        if n < 0 or n > weights.shape[2]:
            out.append(None)
            continue
        sets = []
        for w in np.asarray(weights, np.float64)[s]:
            if n <= keep:
                sets.append(np.arange(n))
                continue
            mid = range(sinks, n - recent)
            best = sorted(mid, key=lambda t: (np.isnan(w[t]), -w[t] if w[t] == w[t] else 0.0, t))[: keep - sinks - recent]
            sets.append(np.array(list(range(sinks)) + sorted(best) + list(range(n - recent, n)), np.int64))
        out.append(sets)
    return out


def compact(k_pool, v_pool, table, page, kept, lengths, new_len, weights=None):
    """Pools and weights after the move (copies; kept [n_seqs][sets])."""
    kp, vp = k_pool.copy(), v_pool.copy()
    w = None if weights is None else weights.copy()
    num_pages = kp.shape[0] // page
    for s, n in enumerate(new_len):
        if n == lengths[s]:
            continue
        for h in range(kp.shape[1]):
            u = 0 if len(kept[s]) == 1 else h
            for i in range(n):
                a, b = (slot_of(table, page, num_pages, s, t) for t in (i, int(kept[s][u][i])))
                if a is not None and b is not None:
                    kp[a, h], vp[a, h] = k_pool[b, h], v_pool[b, h]
        if w is not None:
            for u in range(len(kept[s])):
                for i in range(n):
                    if None not in [slot_of(table, page, num_pages, s, t) for t in (i, int(kept[s][u][i]))]:
                        w[s, u, i] = weights[s, u, int(kept[s][u][i])]
    return kp, vp, w
