"""Plain reference of attention with capped and biased scores, rows' first tokens
and prefixes, in 64 bits and straight from the formula of pq_attn_mod."""
from __future__ import annotations

import numpy as np

import kvref

F32 = np.float32


def attention(cache, row_start, q, n_q, scale, window=0, sinks=0, cap=0.0, slope=None, first=None, prefix=None):
    """(out, vmax); q [n_rows, n_q, d]. vmax: largest |v| that a row and head sees."""
    n_rows, g = q.shape[0], n_q // cache.n_kv
    out, vmax = np.zeros((n_rows, n_q, cache.d)), np.zeros((n_rows, n_q))
    for r, (s, pos) in enumerate(kvref.places(cache, row_start, n_rows)):
        if pos < 0:
            continue
        end = min(max(int(cache.len[s]), 0), cache.table_ld * cache.page)
        t = np.arange(end)
        behind = (t <= pos) & ((window == 0) | (pos - t < window) | (t < sinks))
        see = behind | (t < (int(prefix[r]) if prefix is not None else 0))
        see &= t >= (int(first[r]) if first is not None else 0)
        pg = cache.table[s][t // cache.page]
        see &= (pg >= 0) & (pg < cache.n_pages)
        if not see.any():
            continue
        t, pg = t[see], pg[see]
        for kvh in range(cache.n_kv):
            k = cache.k[pg, kvh, t % cache.page].astype(np.float64) * cache.ks[pg, kvh][:, None].astype(np.float64)
            v = cache.v[pg, kvh, t % cache.page].astype(np.float64) * cache.vs[pg, kvh][:, None].astype(np.float64)
            hs = slice(kvh * g, kvh * g + g)
            x = q[r, hs].astype(np.float64) @ k.T * float(F32(scale))
            if cap:
                x = float(F32(cap)) * np.tanh(x / float(F32(cap)))
            if slope is not None:
                x = x - slope[hs].astype(np.float64)[:, None] * np.abs(pos - t)
            w = np.exp(x - x.max(1, keepdims=True))
            out[r, hs] = (w @ v) / w.sum(1, keepdims=True)
            vmax[r, hs] = np.abs(v).max()
    return out, vmax


def slopes(n_q):
    return (2.0 ** (-8.0 * (np.arange(n_q) + 1) / n_q)).astype(F32)


def documents(cache, row_start, n_rows, mean, prefix, seed):
    """(first, prefix) of every row: documents of mean / 2 .. 2 mean tokens behind each other, the first `prefix` tokens of
    each seen from all of it."""
    rng = np.random.default_rng(seed)
    starts = []
    for s in range(cache.n_seq):
        at = [0]
        while at[-1] < cache.len[s]:
            at.append(at[-1] + int(rng.integers(max(1, mean // 2), 2 * mean)))
        starts.append(np.asarray(at))
    first, end = np.zeros(n_rows, np.int32), np.zeros(n_rows, np.int32)
    for r, (s, pos) in enumerate(kvref.places(cache, row_start, n_rows)):
        if pos < 0:
            continue
        i = int(np.searchsorted(starts[s], pos, side="right")) - 1
        first[r] = starts[s][i]
        stop = starts[s][i + 1] if i + 1 < len(starts[s]) else cache.len[s]
        end[r] = min(starts[s][i] + prefix, stop)
    return first, end
