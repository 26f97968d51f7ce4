"""Plain references for the paged 8-bit cache and the attention over it.

Attention in 64 bits straight from its formula, one row and head at a time;
the append in f32 with the roundings that pq.h states (numpy rounds every
elementwise operation, so codes and scales come out bit for bit).
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


class Cache:
    """A host copy of a cache with the caller's view of it."""

    def __init__(self, n_seq, lens, n_kv, page, d, seed, table_ld=None, spare=2):
        rng = np.random.default_rng(seed)
        self.n_seq, self.n_kv, self.page, self.d = n_seq, n_kv, page, d
        self.len = np.asarray(lens, dtype=np.int32)
        need = [-(-max(int(n), 0) // page) for n in lens]
        self.table_ld = table_ld or max(1, max(need))
        need = [min(m, self.table_ld) for m in need]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((n_seq, self.table_ld), -1, dtype=np.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        shape = (self.n_pages, n_kv, page, d)
        self.k = np.clip(np.round(rng.normal(0, 30, shape)), -127, 127).astype(np.int8)
        self.v = np.clip(np.round(rng.normal(0, 30, shape)), -127, 127).astype(np.int8)
        self.ks = (0.033 * np.exp(0.3 * rng.normal(size=(self.n_pages, n_kv)))).astype(F32)
        self.vs = (0.033 * np.exp(0.3 * rng.normal(size=(self.n_pages, n_kv)))).astype(F32)
        # pages that no table names hold what must never be read
        unused = order[at:]
        self.ks[unused] = np.nan
        self.vs[unused] = np.nan

    def page_at(self, s, pos):
        j = pos // self.page
        if pos < 0 or j >= self.table_ld:
            return -1
        p = int(self.table[s, j])
        return p if 0 <= p < self.n_pages else -1


def places(cache, row_start, n_rows):
    """(sequence, position) of every row."""
    if row_start is None:
        return [(s, int(cache.len[s]) - 1) for s in range(n_rows)]
    out = []
    for s in range(cache.n_seq):
        m = int(row_start[s + 1] - row_start[s])
        out += [(s, int(cache.len[s]) - m + i) for i in range(m)]
    return out


def attention(cache, row_start, q, n_q, scale, window, sinks):
    """(out, vmax) in 64 bits; q [n_rows, n_q, d]. vmax: largest |v| that a row and head sees."""
    n_rows = q.shape[0]
    out = np.zeros((n_rows, n_q, cache.d))
    vmax = np.zeros((n_rows, n_q))
    for r, (s, pos) in enumerate(places(cache, row_start, n_rows)):
        see = [t for t in range(pos + 1)
               if (window == 0 or pos - t < window or t < sinks) and cache.page_at(s, t) >= 0]
        if not see:
            continue
        t = np.asarray(see)
        pg = np.asarray([cache.page_at(s, x) for x in see])
        for kvh in range(cache.n_kv):
            k = cache.k[pg, kvh, t % cache.page].astype(np.float64) * cache.ks[pg, kvh][:, None].astype(np.float64)
            v = cache.v[pg, kvh, t % cache.page].astype(np.float64) * cache.vs[pg, kvh][:, None].astype(np.float64)
            g = n_q // cache.n_kv
            for h in range(kvh * g, kvh * g + g):
                x = k @ q[r, h].astype(np.float64) * float(F32(scale))
                w = np.exp(x - x.max())
                out[r, h] = (w @ v) / w.sum()
                vmax[r, h] = np.abs(v).max()
    return out, vmax


def rotate(x, cos, sin, rot, mode):
    """x [heads, d] f32 at one position; cos, sin [rot/2]."""
    y = x.copy()
    h = rot // 2
    a, b = (x[:, :h], x[:, h:rot]) if mode == "half" else (x[:, 0:rot:2], x[:, 1:rot:2])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    if mode == "half":
        y[:, :h], y[:, h:rot] = ya, yb
    else:
        y[:, 0:rot:2], y[:, 1:rot:2] = ya, yb
    return y


def append(cache, row_start, k, v, cos, sin, rot, mode):
    """Append rows k, v [n_rows, n_kv, d] (f32) to the cache in place."""
    n_rows = k.shape[0]
    blocks = {}
    for r, (s, pos) in enumerate(places(cache, row_start, n_rows)):
        if pos < 0:
            continue
        pg = cache.page_at(s, pos)
        if pg >= 0:
            blocks.setdefault(pg, []).append((r, pos))
    with np.errstate(invalid="ignore", over="ignore"):
        for pg, rows in blocks.items():
            keep = min(pos for _, pos in rows) % cache.page
            for codes, scale, src, turn in ((cache.k, cache.ks, k, True), (cache.v, cache.vs, v, False)):
                new = {}
                for r, pos in rows:
                    x = src[r].astype(F32)
                    if turn and rot:
                        n_pos = cos.shape[0]
                        c = cos[pos] if pos < n_pos else np.full(rot // 2, np.nan, F32)
                        sn = sin[pos] if pos < n_pos else np.full(rot // 2, np.nan, F32)
                        x = rotate(x, c, sn, rot, mode)
                    new[pos] = x
                for h in range(cache.n_kv):
                    vals = np.concatenate([x[h] for x in new.values()])
                    top = F32(np.abs(vals).max()) / F32(127)          # NaN passes through max
                    if not np.isfinite(top):
                        top = F32(np.nan)
                    elif top < F32(2.0 ** -126):
                        top = F32(0)
                    old = scale[pg, h] if keep else F32(0)
                    now = F32(np.nan) if np.isnan(top) or np.isnan(old) else max(top, old)
                    if keep and now > old:
                        was = codes[pg, h, :keep].astype(F32)
                        codes[pg, h, :keep] = np.rint(was * (old / now)).astype(np.int8)
                    inv = F32(1) / now if now > 0 else F32(0)
                    for pos, x in new.items():
                        code = np.rint(x[h] * inv)
                        codes[pg, h, pos % cache.page] = np.where(np.isnan(code), 0, np.clip(code, -127, 127)).astype(np.int8)
                    scale[pg, h] = now


def gather(cache, row_start, n_rows):
    """Values of the rows' tokens, f32 [n_rows, n_kv, d] for K and V."""
    out = [np.zeros((n_rows, cache.n_kv, cache.d), F32) for _ in range(2)]
    for r, (s, pos) in enumerate(places(cache, row_start, n_rows)):
        pg = cache.page_at(s, pos)
        if pg >= 0:
            for o, codes, scale in ((out[0], cache.k, cache.ks), (out[1], cache.v, cache.vs)):
                o[r] = codes[pg, :, pos % cache.page].astype(F32) * scale[pg][:, None]
    return out
