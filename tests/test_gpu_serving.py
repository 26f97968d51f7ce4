"""The pool, the cache and attention with modified scores together, as a serving program runs them: prompts, shared and
sampled, single-token steps, drafts taken back, sequences finished and the pool compacted, over two layers.

Attention is checked against 64 bits on the cache's own values (gathered as f32: scale * code rounded once, 2^-24 of
each, far below the bounds of test_gpu_attn_mod.py, which are used here), and codes against a program that shares
nothing: every sequence of its own, appended to in the same pieces, so that scales and codes are the same.
"""
import numpy as np
import pytest

import quantized_weight_mat_gb300 as pq

pytestmark = pytest.mark.gpu
N_Q, N_KV, D, PAGE = 8, 2, 64, 32
LAYERS, N_SEQ, WIDTH = 2, 8, 12
CAP, POS = 30.0, WIDTH * PAGE


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


class Program:
    """What a serving program keeps, with a pool (n_pages) or with pages of its own for every sequence."""

    def __init__(self, n_pages, pooled):
        import torch
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.pooled, self.n_pages = pooled, n_pages
        self.k = torch.zeros(LAYERS, n_pages, N_KV, PAGE, D, dtype=torch.int8, device="cuda")
        self.v, self.ks = torch.zeros_like(self.k), torch.zeros(LAYERS, n_pages, N_KV, device="cuda")
        self.vs = torch.zeros_like(self.ks)
        self.len, self.refs = z(N_SEQ), z(n_pages)
        self.table = torch.full((N_SEQ, WIDTH), -1, dtype=torch.int32, device="cuda")
        if not pooled:
            self.table.copy_(torch.arange(N_SEQ * WIDTH, dtype=torch.int32).view(N_SEQ, WIDTH))
        self.caches = [pq.pq_kv_cache(self.k[i], self.v[i], self.ks[i], self.vs[i], self.table, self.len, n_pages, N_KV, PAGE, D,
                                      N_SEQ, WIDTH) for i in range(LAYERS)]
        self.layers = pq.pq_kv_layers(self.caches)
        self.pool = pq.pq_kv_pool(self.refs, self.table, self.len, n_pages, PAGE, N_SEQ, WIDTH)
        self.status, self.used = z(2), z(1)
        n = max(pq.pq_kv_pool_ws_bytes(self.pool), pq.pq_attn_mod_ws_bytes(N_Q, N_KV, D, 1024, N_SEQ))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        a = torch.arange(POS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
        self.cos, self.sin = a.cos().float(), a.sin().float()
        slope = torch.tensor([2.0 ** -(i + 1) for i in range(N_Q)], device="cuda")
        self.mods = [pq.pq_score_mod(CAP), pq.pq_score_mod(0.0, slope)]      # a layer with capped scores, one with biased ones

    def tokens(self, news, seed_of, dt="f32"):
        """news[s] tokens appended to each sequence, their q, k and v made from seed_of[s] and the position; attention of both layers."""
        import torch
        n = torch.tensor(news, dtype=torch.int32, device="cuda")
        if self.pooled:
            pq.pq_kv_reserve(self.pool, self.layers, n, self.status, self.ws, self.ws.numel())
            assert self.status.tolist() == [0, 0]
        start = [int(x) for x in self.len.tolist()]
        rows = torch.cat([rows_of(seed_of[s], start[s], m) for s, m in enumerate(news) if m]) if sum(news) else None
        rs = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
        self.len += n
        outs = []
        for i, cache in enumerate(self.caches):
            x = (rows * (i + 1)).to({"f32": torch.float32, "bf16": torch.bfloat16}[dt])
            w = x.shape[1]
            pq.pq_kv_append(cache, rs, x.shape[0], dt, x[:, N_Q * D:], w, x[:, (N_Q + N_KV) * D:], w, x, w, N_Q, x, w, self.cos,
                            self.sin, POS, D, "half")
            out = torch.empty(x.shape[0], N_Q * D, dtype=x.dtype, device="cuda")
            pq.pq_attn_mod(cache, rs, x.shape[0], dt, x, w, N_Q, D ** -0.5, 0, 0, self.mods[i], out, N_Q * D, self.ws, self.ws.numel())
            outs.append((x, out))
        return rs, outs

    def values(self, layer):
        """Keys and values of every sequence."""
        import torch
        got = []
        for s, n in enumerate(self.len.tolist()):
            rs = torch.zeros(N_SEQ + 1, dtype=torch.int32, device="cuda")
            rs[s + 1:] = n
            k = torch.empty(max(n, 1), N_KV * D, device="cuda")
            v = torch.empty_like(k)
            pq.pq_kv_gather(self.caches[layer], rs, n, "f32", k, N_KV * D, v, N_KV * D)
            got.append((k[:n].cpu(), v[:n].cpu()))
        return got


def rows_of(seed, start, m):
    import torch
    return torch.stack([torch.randn((N_Q + 2 * N_KV) * D, generator=torch.Generator().manual_seed(1000 * seed + p)) for p in range(start, start + m)]).cuda()


def check_attention(prog, rs, outs, dt):
    import torch
    for layer, (x, out) in enumerate(outs):
        vals, starts, lens = prog.values(layer), rs.tolist(), prog.len.tolist()
        for s in range(N_SEQ):
            k, v = (t.double().view(-1, N_KV, D) for t in vals[s])
            for r in range(starts[s], starts[s + 1]):
                pos = lens[s] - starts[s + 1] + r
                q = x[r, :N_Q * D].double().cpu().view(N_KV, N_Q // N_KV, D)
                z = torch.einsum("hgd,thd->hgt", q, k[:pos + 1]) * D ** -0.5
                if layer == 0:
                    z = CAP * torch.tanh(z / CAP)
                else:
                    z -= torch.tensor([2.0 ** -(i + 1) for i in range(N_Q)], dtype=torch.float64).view(N_KV, -1, 1) * (pos - torch.arange(pos + 1))
                ref = torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), v[:pos + 1])
                got = out[r].double().cpu().view_as(ref)
                vmax = float(v[:pos + 1].abs().max())
                # scores: sums of |q k| scale log2 e below 64 here (q and k three times as long in the second layer)
                tol = (2 * 64 * 2.0 ** -20 + 2 * 0.6932 * 1.4427 * (2.0 ** -21 * (16 if dt == "f32" else CAP) + 3 * 2.0 ** -24 * 64)) * vmax
                tol = tol + (2.0 ** -11 * vmax + 2.0 ** -8 * ref.abs() if dt == "bf16" else 2.0 ** -24 * ref.abs())
                assert bool(((got - ref).abs() <= tol).all()), (layer, s, r)


def check_pool(prog):
    import torch
    named = prog.table[prog.table >= 0].long()
    assert torch.equal(torch.bincount(named, minlength=prog.n_pages).int(), prog.refs)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_serving_run(dt):
    import torch
    a, b = Program(70, True), Program(N_SEQ * WIDTH, False)
    seeds = list(range(N_SEQ))

    def step(news):
        rs, outs = a.tokens(news, seeds, dt)
        _, alone = b.tokens(news, seeds, dt)
        for (_, x), (_, y) in zip(outs, alone):
            assert torch.equal(x, y)                   # the same codes, wherever they lie
        check_attention(a, rs, outs, dt)
        check_pool(a)

    def same():
        for i in range(LAYERS):
            for (k, v), (k2, v2) in zip(a.values(i), b.values(i)):
                assert torch.equal(k, k2) and torch.equal(v, v2)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def fork(frm, to, tokens=None):
        pq.pq_kv_fork(a.pool, len(to), ints(frm), ints(to), None if tokens is None else ints(tokens), a.ws, a.ws.numel())
        # the program without a pool copies codes instead
        k, v, ks, vs = (t.clone() for t in (b.k, b.v, b.ks, b.vs))
        lens = b.len.clone()
        for i, (f, t) in enumerate(zip(frm, to)):
            for x, was in ((b.k, k), (b.v, v), (b.ks, ks), (b.vs, vs)):
                x[:, t * WIDTH:(t + 1) * WIDTH] = was[:, f * WIDTH:(f + 1) * WIDTH]
            b.len[t] = lens[f] if tokens is None else min(int(lens[f]), tokens[i])
        assert torch.equal(a.len, b.len)
        same()
        check_pool(a)

    # two prompts, one of them sampled three times; a third one begins like the first, by whole pages
    step([70, 0, 0, 0, 45, 0, 0, 0])
    fork([0, 0, 0, 4], [1, 2, 3, 5])
    fork([0], [6], [64])
    for _ in range(3):
        step([1, 1, 1, 1, 1, 1, 30, 0])
    # beams: the second one goes on twice
    fork([1, 1, 0, 2], [0, 1, 2, 3])
    seeds[0], seeds[2] = 20, 21                        # other tokens from here on
    step([1, 1, 1, 1, 0, 0, 0, 0])
    # five drafted tokens, two of them kept
    step([5, 5, 5, 5, 0, 5, 0, 0])
    keep = [n - 3 if s < 4 or s == 5 else n for s, n in enumerate(a.len.tolist())]
    pq.pq_kv_free(a.pool, N_SEQ, None, ints(keep))
    b.len.copy_(ints(keep))
    assert torch.equal(a.len, b.len)
    check_pool(a)
    step([2, 1, 1, 2, 0, 1, 0, 0])
    # two sequences finish, the pool moves together, the rest goes on
    pq.pq_kv_free(a.pool, 2, ints([4, 1]))
    b.len[4] = b.len[1] = 0
    pq.pq_kv_compact(a.pool, a.layers, None, a.used, a.ws, a.ws.numel())
    used = int(a.used[0])
    assert used == int((a.refs > 0).sum()) and int(a.table.max()) < used
    same()
    step([1, 40, 1, 1, 33, 1, 1, 64])
    pq.pq_kv_free(a.pool, N_SEQ)
    assert not a.refs.any() and not a.len.any() and pq.pq_wait_timeouts() == 0
