"""fp64 oracles of the operators around the verify matmul (test infrastructure
only): rotary append, attention over a paged cache, sampling.  Plain loops over
requests, from the definitions in include/lbv.h."""
from __future__ import annotations

import numpy as np


def positions(q_start, kv_len):
    """(request, cache position) of every row; request -1 for rows of none."""
    rows = int(max(q_start))
    req = np.full(rows, -1, np.int64)
    pos = np.zeros(rows, np.int64)
    for r in range(len(kv_len)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        req[a:b] = r
        pos[a:b] = int(kv_len[r]) - (b - a) + np.arange(b - a)
    return req, pos


def rotate(x, pos, freqs, interleaved, factor):
    """x [rows, heads, dim] fp64, rotated by pos [rows] * freqs radians; also the
    sum |a| + |b| of each element's pair (0 where nothing rotates)."""
    half = len(freqs)
    y, size = x.copy(), np.zeros_like(x)
    ang = pos[:, None].astype(np.float64) * np.asarray(freqs, np.float64)[None]
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None]
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def gather(cache, table, page_size, count):
    """Slots 0..count-1 of one request: [count, heads, dim]; pages outside the
    cache read as zeros."""
    out = np.zeros((count,) + cache.shape[2:], np.float64)
    for j in range(count):
        page = int(table[j // page_size])
        if 0 <= page < cache.shape[0]:
            out[j] = cache[page, j % page_size]
    return out


def attend(q, k_cache, v_cache, q_start, kv_len, table, scale, window=0, tree=None):
    """Returns out, lse, and what tolerances are made of: A = sum p |v| / sum p,
    V = sum |v| / sum 2^(t - max t), S = max_j scale sum |q_d k_d|."""
    rows, heads, dim = q.shape
    ps, hk = k_cache.shape[1], k_cache.shape[2]
    g = heads // hk
    out, A, V = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    lse, S = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    for r in range(len(kv_len)):
        a, b = int(q_start[r]), int(q_start[r + 1])
        n, kv = b - a, int(kv_len[r])
        keys = max(0, min(kv, table.shape[1] * ps))
        k, v = gather(k_cache, table[r], ps, keys), gather(v_cache, table[r], ps, keys)
        first = kv - n
        j = np.arange(keys)
        for i in range(n):
            if tree is None:
                see = j <= first + i
            else:
                w = int(tree[a + i]) & (2**64 - 1)
                bit = np.array([(w >> int(x)) & 1 if 0 <= x < 64 else 0 for x in j - first], bool)
                see = (j < first) | bit
            if window:
                see = see & (j > first + i - window)
            if not see.any():
                continue
            for h in range(heads):
                kk, vv = k[see, h // g], v[see, h // g]
                t = kk @ q[a + i, h] * scale
                p = np.exp(t - t.max())
                lse[a + i, h] = t.max() + np.log(p.sum())
                out[a + i, h] = p @ vv / p.sum()
                A[a + i, h] = p @ np.abs(vv) / p.sum()
                V[a + i, h] = np.abs(vv).sum(0) / p.sum()
                S[a + i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[a + i, h])).max()
    return out, lse, A, V, S


def sample_sets(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, last=False, slack=0.0):
    """Kept tokens of one row of fp64 logits (masked ones -inf), in rank order,
    with the top-p and min-p bounds moved by a relative `slack`; and their
    drawing weights.  Greedy rows keep the first maximum."""
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if order.size == 0:
        return order, np.zeros(0)
    z = np.zeros(order.size)
    same = x[order] == x[order[0]]
    z[~same] = x[order][~same] - x[order[0]]
    if not temperature > 0:
        return order[:1], np.ones(1)
    w = np.exp(z if last else z / temperature)
    n = min(order.size, top_k) if top_k > 0 else order.size
    keep = np.arange(order.size) < n
    if top_p < 1:
        before = np.cumsum(w) - w
        share = np.floor(top_p * 2**24) / 2**24
        keep &= before < (share + slack) * w[:n].sum()
    if min_p > 0:
        keep &= w >= min_p * (1 - slack)
    keep[0] = True
    return order[keep], np.exp(z / temperature)[keep]
