"""Attention with capped scores, a bias by distance, documents and prefixes, against 64 bits (tests/modref.py).

Bounds as in test_gpu_attn.py, where a weight is off by a relative 2 ln 2 of the error of its score times log2 e.  That
error grows by (pq.h, pq_attn_mod) the cap's, 2^-21 of the cap, or of a score below 16 for f32 rows, times log2 e; and by
the bias's, three roundings (of the slope times log2 e, of the sum and of its difference from the maximum) of a bias that
is at most 64 above the row's smallest (a larger one leaves a weight below e^-48), 2^-24 of 64 log2 e each.  A case in which
every token is far away adds 2^-24 of that bias each.
"""
import numpy as np
import pytest

import kvref
import modref
import quantized_weight_mat_gb300 as pq
from test_gpu_attn import DTS, HEADS, ws  # noqa: F401
from test_gpu_kv_cache import tdt, upload

pytestmark = pytest.mark.gpu
LOG2E = 1.4427


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


def run(c, news, dt, n_q, ws, window=0, sinks=0, cap=0.0, slope=None, first=None, prefix=None, qmul=1.0, pad=16, far=0.0, seed=1):
    import torch
    row_start = None if news is None else np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n_rows = c.n_seq if news is None else int(row_start[-1])
    w, scale = n_q * c.d, c.d ** -0.5
    q = torch.from_numpy(np.random.default_rng(seed).normal(0, qmul, (n_rows, w + pad)).astype(np.float32)).to(tdt(dt)).cuda()
    t, h = upload(c)
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    mod = pq.pq_score_mod(cap, dev(slope), dev(first), dev(prefix))
    out = torch.full((n_rows + 1, w + 8), 99.0, dtype=tdt(dt), device="cuda")
    size = pq.pq_attn_mod_ws_bytes(n_q, c.n_kv, c.d, n_rows, c.n_seq)
    assert 0 < size <= ws.numel()
    args = (h, dev(row_start), n_rows, dt, q, w + pad, n_q, scale, window, sinks, mod, out, w + 8, ws, size)
    pq.pq_attn_mod(*args)
    torch.cuda.synchronize()
    assert torch.all(out[n_rows] == 99.0) and torch.all(out[:, w:] == 99.0)
    got = out[:n_rows, :w].clone()
    out.fill_(99.0)                                # bit for bit the same, from what the first call left in ws
    pq.pq_attn_mod(*args)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.uint8), out[:n_rows, :w].contiguous().view(torch.uint8))
    qf = q.float().cpu().numpy()[:, :w].reshape(n_rows, n_q, c.d)
    ref, vmax = modref.attention(c, row_start, qf, n_q, scale, window, sinks, cap, slope, first, prefix)
    got = got.float().cpu().numpy().reshape(n_rows, n_q, c.d)
    off = 0.0
    if cap:
        off += 2.0 ** -21 * LOG2E * (16 if dt == "f32" else cap)
    if slope is not None:
        off += 3 * 2.0 ** -24 * LOG2E * (64 + far)
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    tol = (4e-5 + 2 * 0.6932 * off + (2.0 ** -11 if dt != "f32" else 0.0)) * vmax[..., None] + u * np.abs(ref) + 1e-30
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound"
    assert (got[vmax == 0] == 0).all()             # rows that see nothing


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 0, 1000]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("cap,bias", [(2.0, False), (50.0, False), (0.0, True), (5.0, True)])
def test_one_token_each(dt, heads, cap, bias, ws):  # noqa: F811
    n_q, n_kv, d = heads
    c = kvref.Cache(len(LENS), LENS, n_kv, 16 if bias else 64, d, seed=d)
    run(c, None, dt, n_q, ws, cap=cap, slope=modref.slopes(n_q) if bias else None)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("news", [[5, 1, 0, 5, 3], [40, 1, 0, 40, 21], [270, 3, 0, 100, 190]])
@pytest.mark.parametrize("what", ["cap", "bias", "both"])
def test_several_tokens(dt, heads, news, what, ws):  # noqa: F811
    n_q, n_kv, d = heads
    if news[0] > 40 and d not in (64, 128):
        news = [min(m, 60) for m in news]
    lens = [news[0], 70, 40, 100 + news[3], 333]
    c = kvref.Cache(len(lens), lens, n_kv, 32, d, seed=news[0])
    run(c, news, dt, n_q, ws, cap=0.0 if what == "bias" else 10.0, slope=None if what == "cap" else modref.slopes(n_q))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (4, 2, 96)])
@pytest.mark.parametrize("news", [None, [7, 3, 0, 20], [300, 1, 0, 150]])
@pytest.mark.parametrize("mean,prefix,window,sinks", [(40, 0, 0, 0), (40, 9, 0, 0), (500, 100, 0, 0), (90, 30, 25, 4), (90, 0, 200, 100), (2, 1, 3, 0)])
def test_documents(dt, heads, news, mean, prefix, window, sinks, ws):  # noqa: F811
    n_q, n_kv, d = heads
    lens = [310, 150, 0, 700]
    c = kvref.Cache(len(lens), lens, n_kv, 16, d, seed=mean)
    row_start = None if news is None else np.concatenate([[0], np.cumsum(news)])
    first, end = modref.documents(c, row_start, 4 if news is None else sum(news), mean, prefix, seed=mean)
    run(c, news, dt, n_q, ws, window=window, sinks=sinks, first=first, prefix=end if prefix else None)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [7, 3, 0, 20], [300, 1, 0, 150]])
@pytest.mark.parametrize("prefix,window,bias", [(64, 0, False), (300, 0, True), (200, 50, False), (5, 1, True), (10 ** 6, 0, True)])
def test_one_prefix(dt, news, prefix, window, bias, ws):  # noqa: F811
    lens = [310, 150, 0, 700]
    c = kvref.Cache(len(lens), lens, 2, 64, 128, seed=prefix % 100)
    n = 4 if news is None else sum(news)
    run(c, news, dt, 8, ws, window=window, prefix=np.full(n, prefix, np.int32), slope=modref.slopes(8) if bias else None)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(8, 2, 128), (3, 1, 48)])
@pytest.mark.parametrize("news", [None, [4, 9, 30, 33], [200, 100, 3, 290]])
def test_any_bounds_in_any_order(dt, heads, news, ws):  # noqa: F811
    # rows that see nothing, bounds past the end, below 0, at the ends of 32 bits
    n_q, n_kv, d = heads
    lens = [310, 100, 40, 700]
    c = kvref.Cache(len(lens), lens, n_kv, 32, d, seed=3)
    n = 4 if news is None else sum(news)
    rng = np.random.default_rng(n)
    odd = np.array([-2 ** 31, -1, 0, 1, 2 ** 31 - 1, 10 ** 6], np.int64)
    first = np.where(rng.random(n) < 0.2, rng.choice(odd, n), rng.integers(0, 720, n)).astype(np.int32)
    prefix = np.where(rng.random(n) < 0.2, rng.choice(odd, n), rng.integers(0, 720, n)).astype(np.int32)
    run(c, news, dt, n_q, ws, first=first, prefix=prefix, cap=20.0)
    run(c, news, dt, n_q, ws, first=first, window=60, sinks=40, slope=modref.slopes(n_q), far=700.0)
    run(c, news, dt, n_q, ws, prefix=prefix, window=60, sinks=40)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [30, 5], [260, 290]])
def test_missing_pages_and_rows_before_the_cache(dt, news, ws):  # noqa: F811
    lens = [200, 290] if news else [200, 0]
    c = kvref.Cache(2, lens, 2, 16, 128, seed=8)
    rng = np.random.default_rng(8)
    for j in rng.permutation(c.table_ld)[:c.table_ld // 2]:
        c.table[rng.integers(0, 2), j] = rng.choice([-1, -7, c.n_pages, 2 ** 31 - 1])
    n = 2 if news is None else sum(news)
    run(c, news, dt, 4, ws, cap=30.0, slope=modref.slopes(4), prefix=np.full(n, 33, np.int32), far=150.0)
    run(c, news, dt, 4, ws, window=70, sinks=20, first=np.full(n, 11, np.int32))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [300]])
def test_slopes_of_any_sign_and_size(dt, news, ws):  # noqa: F811
    c = kvref.Cache(1, [700], 2, 32, 64, seed=9)
    # a negative slope favours far tokens: the maximum rises all the way; 100 leaves the nearest token alone
    run(c, news, dt, 8, ws, slope=np.array([-0.5, -0.01, 0.0, 100.0, 1e-6, 1.0, -3.0, 1e4], np.float32), far=2100.0)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [40], [300]])
@pytest.mark.parametrize("cap", [2.0 ** -60, 0.01, 1.0, 2.0 ** 60])
def test_caps_of_any_size(dt, news, cap, ws):  # noqa: F811
    # scores far past the cap are all the cap; a large one changes nothing beside its own error, which the bound has
    c = kvref.Cache(1, [700], 2, 32, 128, seed=10)
    if cap > 2.0 ** 20 and dt != "f32":
        return
    run(c, news, dt, 8, ws, cap=cap, qmul=1.0 if cap > 1 else 5.0)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows", [1, 6, 300])
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64), (4, 2, 80)])
def test_without_mods_it_is_pq_attn(dt, rows, heads, ws):  # noqa: F811
    import torch
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 32, d, seed=11)
    _, h = upload(c)
    w = n_q * d
    q = torch.randn(rows, w, device="cuda").to(tdt(dt))
    rs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    outs = [torch.empty(rows, w, dtype=q.dtype, device="cuda") for _ in range(3)]
    tail = (rs, rows, dt, q, w, n_q, 0.1, 100, 4)
    pq.pq_attn(h, *tail, outs[0], w, ws, ws.numel())
    pq.pq_attn_mod(h, *tail, None, outs[1], w, ws, ws.numel())
    pq.pq_attn_mod(h, *tail, pq.pq_score_mod(), outs[2], w, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [270, 33]])
def test_hidden_pages_may_hold_nan(dt, news, ws):  # noqa: F811
    # tokens before a document's first one lie in pages of NaN scales
    c = kvref.Cache(2, [400, 300], 2, 16, 128, seed=12)
    for s in range(2):
        c.ks[c.table[s, :4]] = np.nan
        c.vs[c.table[s, :4]] = np.inf
    n = 2 if news is None else sum(news)
    first = np.full(n, 64, np.int32)
    run(c, news, dt, 4, ws, first=first, cap=10.0)
    run(c, news, dt, 4, ws, first=first, slope=modref.slopes(4), window=90, sinks=70)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64)])
@pytest.mark.parametrize("news", [None, [40], [300]])
@pytest.mark.parametrize("what", ["cap", "bias"])
def test_scales_of_very_different_pages(dt, heads, news, what, ws):  # noqa: F811
    # pages of key scales from tiny to so large that their scores are all far beyond the cap, zero keys among them
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 32, d, seed=14)
    rng = np.random.default_rng(14)
    named = c.table[0]
    c.vs[named] *= 10.0 ** rng.integers(-6, 3, (len(named), n_kv))
    if what == "cap":
        c.ks[named[::3]] *= 1e12
        c.ks[named[1::5]] *= 1e-9
        c.k[named[::6]] = 0
        run(c, news, dt, n_q, ws, cap=3.0)
        run(c, news, dt, n_q, ws, cap=2.0 ** -60)
    else:
        run(c, news, dt, n_q, ws, slope=modref.slopes(n_q))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows", [1, 40])
def test_long_contexts(dt, rows, ws):  # noqa: F811
    # one row tile shared by many CTAs, from the row's own token back; documents that begin far into the sequence
    n = 20000
    c = kvref.Cache(1, [n], 2, 64, 64, seed=15)
    news = None if rows == 1 else [rows]
    run(c, news, dt, 8, ws, slope=modref.slopes(8) / 16)
    run(c, news, dt, 8, ws, cap=20.0, first=np.full(rows, 9000, np.int32), prefix=np.full(rows, 9100, np.int32), window=3000)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_streams_with_a_workspace_each(dt):
    import torch
    c = kvref.Cache(3, [900, 400, 150], 2, 32, 128, seed=16)
    _, h = upload(c)
    rs = torch.tensor([0, 300, 500, 510], dtype=torch.int32, device="cuda")
    slope = torch.from_numpy(modref.slopes(8)).cuda()
    first = torch.full((510,), 50, dtype=torch.int32, device="cuda")
    mods = [pq.pq_score_mod(20.0, None, first), pq.pq_score_mod(0.0, slope)]
    qs = [torch.randn(510, 1024, device="cuda").to(tdt(dt)) for _ in mods]
    size = pq.pq_attn_mod_ws_bytes(8, 2, 128, 510, 3)
    wss = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in mods]

    def call(i, out, stream=None):
        pq.pq_attn_mod(h, rs, 510, dt, qs[i], 1024, 8, 0.1, 0, 0, mods[i], out, 1024, wss[i], size, stream=stream)

    want = [torch.empty_like(q) for q in qs]
    for i in (0, 1):
        call(i, want[i])
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in mods], [[torch.empty_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for k in range(20):
        for i in (0, 1):
            call(i, outs[i][k], streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in outs[i])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64), (4, 2, 80)])
@pytest.mark.parametrize("news", [None, [40], [300]])
@pytest.mark.parametrize("what", ["ks", "vs", "q"])
def test_nan_reaches_the_rows_that_see_it(dt, heads, news, what, ws):  # noqa: F811
    # a NaN behind the cap and beside the bias: all of the rows that see it, none of the others
    import torch
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 32, d, seed=17)
    n = 1 if news is None else news[0]
    pos = np.arange(700 - n, 700)
    if what != "q":
        getattr(c, what)[c.table[0, 20], 1] = np.nan       # tokens 640 to 671 of the second kv head
    first = np.where(np.arange(n) % 3 == 0, 672, 0).astype(np.int32)
    first = np.minimum(first, pos).astype(np.int32)
    _, h = upload(c)
    q = torch.randn(n, n_q * d, device="cuda").to(tdt(dt))
    if what == "q":
        q[n // 2, 5] = float("nan")                        # the first query head of one row
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    rs = None if news is None else torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for mod in (pq.pq_score_mod(5.0, None, dev(first)), pq.pq_score_mod(0.0, dev(modref.slopes(n_q)), dev(first)),
                pq.pq_score_mod(5.0, dev(modref.slopes(n_q)), dev(first))):
        out = torch.zeros_like(q)
        pq.pq_attn_mod(h, rs, n, dt, q, n_q * d, n_q, d ** -0.5, 0, 0, mod, out, n_q * d, ws, ws.numel())
        torch.cuda.synchronize()
        nan = out.float().cpu().isnan().view(n, n_q, d).numpy()
        want = np.zeros((n, n_q, d), bool)
        if what == "q":
            want[n // 2, 0] = True
        else:
            want[(first < 672) & (pos >= 640), n_q // n_kv:] = True
        assert np.array_equal(nan, want)


@pytest.mark.parametrize("news", [None, [257, 1]])
def test_in_a_cuda_graph_with_bounds_that_move(news, ws):  # noqa: F811
    import torch
    c = kvref.Cache(2, [500, 300], 2, 32, 128, seed=13)
    t, h = upload(c)
    n, n_q, w = (2 if news is None else sum(news)), 8, 8 * 128
    rs = None if news is None else torch.tensor([0, news[0], n], dtype=torch.int32, device="cuda")
    q = torch.randn(n, w, device="cuda").bfloat16()
    first = torch.zeros(n, dtype=torch.int32, device="cuda")
    slope = torch.from_numpy(modref.slopes(n_q)).cuda()
    mod = pq.pq_score_mod(30.0, slope, first, None)
    out = torch.empty_like(q)
    args = (h, rs, n, "bf16", q, w, n_q, 0.1, 0, 0, mod, out, w, ws, ws.numel())
    pq.pq_attn_mod(*args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.pq_attn_mod(*args)
    for lens, f in (([500, 300], 10), ([450, 299], 40), ([300, 270], 299)):
        t["len"].copy_(torch.tensor(lens, dtype=torch.int32))
        first.fill_(f)
        g.replay()
        got = out.clone()
        out.zero_()
        pq.pq_attn_mod(*args)
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_no_wait_ran_out():
    assert pq.pq_wait_timeouts() == 0
