"""Attention over the paged 8-bit cache on the GPU, against 64 bits (tests/kvref.py).

Bounds, per output element, from the kernels' roundings.  Weights p_t / sum are
off by a relative 2 * delta where delta is the error of a score: f32 sums of at
most 256 products and the exponential, below 2^-20 of sum |q k| scale log2 e,
which is under 16 for these inputs: 2 * 16 * 2^-20 < 4e-5.  16-bit rows: the
weights enter the products in 11 bits (2^-11 relative each), and the output is
rounded once: 2^-11 (f16) or 2^-8 (bf16) of itself.  So
    |out - ref| <= (4e-5 [+ 2^-11]) * max|v| + u * |ref|.
"""
import numpy as np
import pytest

import kvref
import quantized_weight_mat_gb300 as pq
from test_gpu_kv_cache import tdt, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def ws():
    import torch
    return torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")


def run(c, news, dt, n_q, ws, window=0, sinks=0, scale=None, seed=1, qmul=1.0, pad=16, twice=True, q=None):
    import torch
    row_start = None if news is None else np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n_rows = c.n_seq if news is None else int(row_start[-1])
    w = n_q * c.d
    scale = c.d ** -0.5 if scale is None else scale
    if q is None:
        q = torch.from_numpy(np.random.default_rng(seed).normal(0, qmul, (n_rows, w + pad)).astype(np.float32))
    q = q.to(tdt(dt)).cuda()
    _, h = upload(c)
    rs = None if news is None else torch.from_numpy(row_start).cuda()
    out = torch.full((n_rows + 1, w + 8), 99.0, dtype=tdt(dt), device="cuda")
    size = pq.pq_attn_ws_bytes(n_q, c.n_kv, c.d)
    assert 0 < size <= ws.numel()
    args = (h, rs, n_rows, dt, q, w + pad, n_q, scale, window, sinks, out, w + 8, ws, size)
    pq.pq_attn(*args)
    torch.cuda.synchronize()
    assert torch.all(out[n_rows] == 99.0) and torch.all(out[:, w:] == 99.0)
    got = out[:n_rows, :w].clone()
    if twice:                                      # bit for bit the same, from what the first call left in ws
        out.fill_(99.0)
        pq.pq_attn(*args)
        torch.cuda.synchronize()
        a, b = got.view(torch.uint8), out[:n_rows, :w].contiguous().view(torch.uint8)
        assert torch.equal(a, b)
    qf = q.float().cpu().numpy()[:, :w].reshape(n_rows, n_q, c.d)
    ref, vmax = kvref.attention(c, row_start, qf, n_q, scale, window, sinks)
    return got.float().cpu().numpy().reshape(n_rows, n_q, c.d), ref, vmax


def check(got, ref, vmax, dt):
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    tol = (4e-5 + (2.0 ** -11 if dt != "f32" else 0.0)) * vmax[..., None] + u * np.abs(ref) + 1e-30
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound"


DTS = ["f32", "f16", "bf16"]
HEADS = [(32, 8, 128), (14, 2, 64), (4, 4, 128), (16, 1, 64), (6, 2, 80), (2, 1, 256)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_one_token_each(dt, heads, page, ws):
    n_q, n_kv, d = heads
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 0, 1000]
    c = kvref.Cache(len(lens), lens, n_kv, page, d, seed=d + page)
    check(*run(c, None, dt, n_q, ws), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("n", [1, 700, 5000])
def test_one_sequence_is_split(dt, page, n, ws):
    c = kvref.Cache(1, [n], 8, page, 128, seed=n)
    check(*run(c, None, dt, 32, ws), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("new", [2, 5, 33])
def test_several_tokens(dt, heads, new, ws):
    n_q, n_kv, d = heads
    news = [new, 1, 0, new, max(1, new // 2)]
    lens = [new, 70, 40, 100 + new, 333]
    c = kvref.Cache(len(lens), lens, n_kv, 32, d, seed=new)
    check(*run(c, news, dt, n_q, ws), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64)])
@pytest.mark.parametrize("lens,news", [([150], [150]), ([400, 1, 260], [129, 1, 260]), ([513], [257]), ([300, 0, 90, 128], [300, 0, 45, 128])])
def test_prompts(dt, heads, lens, news, ws):
    n_q, n_kv, d = heads
    c = kvref.Cache(len(lens), lens, n_kv, 64 if lens[0] != 400 else 16, d, seed=sum(lens))
    check(*run(c, news, dt, n_q, ws), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("n_seq", [5, 40])
def test_sequences_of_several_row_tiles(dt, n_seq, ws):
    # f32: 5 to 8 row tiles each, counted lane by lane or all lanes together
    rng = np.random.default_rng(n_seq)
    news = [int(x) for x in rng.integers(17, 31, n_seq)]
    lens = [m + int(x) for m, x in zip(news, rng.integers(0, 40, n_seq))]
    news[n_seq // 2], lens[n_seq // 2] = 0, 9
    news[1], lens[1] = 150, 170
    c = kvref.Cache(n_seq, lens, 2, 32, 64, seed=31)
    got, ref, vmax = run(c, news, dt, 8, ws)
    check(got, ref, vmax, dt)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (64, 70), (100, 17), (500, 3), (100000, 5), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("news", [None, [3, 1, 40, 150, 0]])
def test_window_and_first_tokens(dt, window, sinks, news, ws):
    lens = [3, 90, 300, 700, 0]
    c = kvref.Cache(len(lens), lens, 2, 16, 64, seed=window % 1000)
    check(*run(c, news, dt, 6, ws, window=window, sinks=sinks), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [4, 3, 170]])
def test_pages_out_of_the_window_may_be_gone(dt, news, ws):
    # pages behind the window were given back: their entries say -1, or point at pages that hold NaN scales
    lens, page, window, sinks = [600, 333, 900], 32, 100, 5
    c = kvref.Cache(3, lens, 2, page, 128, seed=77)
    for s, n in enumerate(lens):
        m = 1 if news is None else news[s]
        lo = max(0, n - m - window + 1) // page
        for j in range(1, lo):
            c.table[s, j] = -1 if j % 2 else c.table[s, j]
            if j % 2 == 0:
                c.ks[c.table[s, j]] = np.nan
                c.vs[c.table[s, j]] = np.inf
    check(*run(c, news, dt, 8, ws, window=window, sinks=sinks), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [70, 2, 200]])
def test_missing_pages_and_short_tables(dt, news, ws):
    lens, page = [100, 90, 250], 16
    c = kvref.Cache(3, lens, 2, page, 64, seed=5, table_ld=12)       # the third sequence is longer than its table
    c.table[0, 1] = -7
    c.table[0, 4] = c.n_pages
    c.table[1, :] = -1                                               # a row that sees nothing
    got, ref, vmax = run(c, news, dt, 4, ws)
    check(got, ref, vmax, dt)
    first = 1 if news is None else 70
    rows = slice(first, first + (1 if news is None else 2))
    assert (got[rows] == 0).all()


@pytest.mark.parametrize("dt", DTS)
def test_more_rows_than_tokens(dt, ws):
    # positions below 0 see nothing
    c = kvref.Cache(2, [3, 140], 2, 16, 64, seed=6)
    got, ref, vmax = run(c, [10, 150], dt, 4, ws)
    check(got, ref, vmax, dt)
    assert (got[:7] == 0).all() and (got[10:20] == 0).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 2, 128), (4, 2, 48)])
@pytest.mark.parametrize("news", [None, [150, 3]])
def test_scores_far_beyond_the_last_bit_of_the_maximum(dt, heads, news, ws):
    # scores up to about 1e11, where one step of an f32 is thousands: the output is v of the largest one
    lens = [400, 37]
    n_q, n_kv, d = heads
    c = kvref.Cache(2, lens, n_kv, 32, d, seed=21)
    got, ref, vmax = run(c, news, dt, n_q, ws, qmul=1e4, scale=1e6)
    assert np.isfinite(got).all()
    import torch
    row_start = None if news is None else np.concatenate([[0], np.cumsum(news)])
    n_rows = c.n_seq if news is None else int(row_start[-1])
    w = n_q * d
    q = torch.from_numpy(np.random.default_rng(1).normal(0, 1e4, (n_rows, w + 16)).astype(np.float32)).to(tdt(dt)).float().numpy()
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    seen = 0
    for r, (s, pos) in enumerate(kvref.places(c, row_start, n_rows)):
        t = np.arange(pos + 1)
        pg = c.table[s, t // c.page]
        for h in range(n_q):
            kvh = h // (n_q // n_kv)
            k = c.k[pg, kvh, t % c.page].astype(np.float64) * c.ks[pg, kvh][:, None]
            parts = np.abs(k * q[r, h * d:(h + 1) * d].astype(np.float64)).sum(axis=1).max()
            x = k @ q[r, h * d:(h + 1) * d].astype(np.float64)
            top = np.sort(x)[-2:]
            # f32 sums of d products: not decided where the two largest are this close
            if len(x) > 1 and top[1] - top[0] < 2.0 ** -16 * parts:
                continue
            seen += 1
            at = int(np.argmax(x))
            v = c.v[pg[at], kvh, at % c.page].astype(np.float64) * c.vs[pg[at], kvh]
            assert (np.abs(got[r, h] - v) <= (4e-5 + (2.0 ** -11 if dt != "f32" else 0.0)) * np.abs(v).max() + u * np.abs(v)).all()
    assert seen > 0.9 * n_rows * n_q


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [150, 3]])
def test_one_token_takes_all(dt, news, ws):
    # scores far apart (up to about 1e4): the softmax is one token, and nothing overflows
    lens = [400, 37]
    c = kvref.Cache(2, lens, 2, 32, 64, seed=9)
    got, ref, vmax = run(c, news, dt, 4, ws, qmul=3000.0)
    # the scores' error grows with q: where a second token comes within 2^-20 of 16 * 3000 * 2, weights may move
    far = np.abs(got - ref) > 1e-2 * vmax[..., None]
    assert np.isfinite(got).all() and far.mean() < 0.02


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [140, 3]])
@pytest.mark.parametrize("amount", [0.0, 1e-30, 1e30])
def test_tiny_and_huge_queries(dt, news, amount, ws):
    if dt == "f16" and amount == 1e30:
        pytest.skip("not an f16 value")
    lens = [300, 37]
    c = kvref.Cache(2, lens, 2, 32, 64, seed=10)
    scale = 0.125 if amount < 1 else 0.125e-30
    got, ref, vmax = run(c, news, dt, 4, ws, qmul=amount, scale=scale)
    check(got, ref, vmax, dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [160, 140]])
def test_scales_of_very_different_pages(dt, news, ws):
    # V scales from 1e-12 to 1e3 and zeros from page to page
    lens = [333, 200]
    c = kvref.Cache(2, lens, 2, 16, 128, seed=14)
    rng = np.random.default_rng(3)
    used = c.table[c.table >= 0]
    c.vs[used] = 10.0 ** rng.uniform(-12, 3, (len(used), 2))
    c.vs[used[::5]] = 0.0
    c.ks[used[1::7]] = 0.0
    check(*run(c, news, dt, 8, ws), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("news", [None, [140, 100]])
def test_nan_scale_reaches_the_rows_that_see_it(dt, news, ws):
    import torch
    lens = [200, 150]
    c = kvref.Cache(2, lens, 2, 16, 64, seed=15)
    c.vs[c.table[0, 5], 1] = np.nan                   # tokens 80..95 of the first sequence, second kv head
    got, ref, _ = run(c, news, dt, 4, ws)
    pos = [p for _, p in kvref.places(c, None if news is None else np.array([0, 140, 240]), got.shape[0])]
    seq = [s for s, _ in kvref.places(c, None if news is None else np.array([0, 140, 240]), got.shape[0])]
    for r in range(got.shape[0]):
        for h in range(4):
            hit = seq[r] == 0 and pos[r] >= 80 and h >= 2
            assert np.isnan(got[r, h]).all() if hit else np.isfinite(got[r, h]).all(), (r, h)


def test_mixed_lengths_over_many_sequences(ws):
    lens = [(i * 131) % 700 for i in range(150)]
    c = kvref.Cache(150, lens, 2, 16, 64, seed=16)
    check(*run(c, None, "bf16", 8, ws), "bf16")
    news = [min(n, 1 + i % 5) for i, n in enumerate(lens)]
    check(*run(c, news, "f16", 8, ws), "f16")


def test_offsets_past_32_bits(ws):
    import torch
    n_kv, page, d, n = 8, 64, 128, 200
    n_pages = 2 ** 31 // (n_kv * page * d) + 64
    small = kvref.Cache(1, [n], n_kv, page, d, seed=18, spare=0)
    k = torch.zeros(n_pages, n_kv, page, d, dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.full((n_pages, n_kv), float("nan"), device="cuda")
    vs = torch.full_like(ks, float("nan"))
    m = small.n_pages
    for big, part in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
        big[n_pages - m:] = torch.from_numpy(part).cuda()
    table = torch.from_numpy(small.table + (n_pages - m)).cuda()
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    h = pq.pq_kv_cache(k, v, ks, vs, table, ln, n_pages, n_kv, page, d, 1, table.shape[1])
    for dt, rows in (("f32", 1), ("bf16", 1), ("bf16", 130)):
        q = torch.randn(rows, 32 * d, device="cuda").to(tdt(dt))
        out = torch.empty_like(q)
        rs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        pq.pq_attn(h, rs, rows, dt, q, 32 * d, 32, d ** -0.5, 0, 0, out, 32 * d, ws, ws.numel(), stream=side)
        side.synchronize()
        ref, vmax = kvref.attention(small, np.array([0, rows]), q.float().cpu().numpy().reshape(rows, 32, d), 32, d ** -0.5, 0, 0)
        check(out.float().cpu().numpy().reshape(rows, 32, d), ref, vmax, dt)


def test_in_a_cuda_graph_with_lengths_that_move(ws):
    import torch
    c = kvref.Cache(3, [64, 300, 500], 2, 32, 128, seed=19)
    t, h = upload(c)
    q = torch.randn(3, 8 * 128, device="cuda")
    out = torch.empty_like(q)

    def step():
        pq.pq_attn(h, None, 3, "f32", q, 1024, 8, 128 ** -0.5, 0, 0, out, 1024, ws, ws.numel())
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([64, 300, 500], [1, 17, 499], [0, 256, 33]):
        c.len[:] = lens
        t["len"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref, vmax = kvref.attention(c, None, q.cpu().numpy().reshape(3, 8, 128), 8, 128 ** -0.5, 0, 0)
        check(out.cpu().numpy().reshape(3, 8, 128), ref, vmax, "f32")


def test_no_rows(ws):
    import torch
    c = kvref.Cache(1, [5], 1, 16, 64, seed=1)
    _, h = upload(c)
    q = torch.zeros(1, 64, device="cuda")
    out = torch.ones(1, 64, device="cuda")
    rs = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert pq.pq_attn(h, rs, 0, "f32", q, 64, 1, 1.0, 0, 0, out, 64, ws, ws.numel()) == 0
    torch.cuda.synchronize()
    assert torch.all(out == 1)


def dense64(t, c, q, n_q, pos, window=0, sinks=0):
    """64-bit attention of the rows of one sequence on the GPU; returns (out, max|v|)."""
    import torch
    n = int(c.len[0])
    tok = torch.arange(n, device="cuda")
    pg = t["table"][0, tok // c.page].long()
    hide = tok > pos[:, None]
    if window:
        hide = hide | ((pos[:, None] - tok >= window) & (tok >= sinks))
    out = torch.empty(q.shape[0], n_q, c.d, dtype=torch.float64, device="cuda")
    vmax = 0.0
    for h in range(c.n_kv):
        k = t["k"][pg, h, tok % c.page].double() * t["ks"][pg, h].double()[:, None]
        v = t["v"][pg, h, tok % c.page].double() * t["vs"][pg, h].double()[:, None]
        vmax = max(vmax, float(v.abs().max()))
        for j in range(h * n_q // c.n_kv, (h + 1) * n_q // c.n_kv):
            x = (q.double()[:, j] @ k.T * float(np.float32(c.d ** -0.5))).masked_fill(hide, -float("inf"))
            out[:, j] = torch.softmax(x, -1) @ v
    return out, vmax


@pytest.mark.parametrize("dt,rows,n,heads,window,sinks", [
    ("bf16", 1, 25001, (32, 8, 128), 0, 0), ("f16", 1, 30000, (14, 2, 64), 0, 0), ("f32", 1, 20011, (16, 1, 64), 0, 0),
    ("f32", 9, 9000, (8, 2, 128), 0, 0), ("bf16", 700, 3100, (32, 8, 128), 0, 0), ("f16", 1500, 1500, (14, 2, 64), 0, 0),
    ("bf16", 64, 30000, (8, 1, 128), 0, 0), ("f16", 900, 5000, (8, 2, 128), 500, 130), ("bf16", 9, 50000, (32, 8, 128), 20000, 7),
])
def test_long_contexts(dt, rows, n, heads, window, sinks, ws):
    import torch
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [n], n_kv, 64, d, seed=rows)
    t, h = upload(c)
    q = torch.randn(rows, n_q * d, device="cuda", generator=torch.Generator("cuda").manual_seed(rows)).to(tdt(dt))
    out = torch.empty_like(q)
    rs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ws.fill_(0xA5)                                    # what the workspace holds does not matter
    pq.pq_attn(h, rs, rows, dt, q, n_q * d, n_q, d ** -0.5, window, sinks, out, n_q * d, ws, ws.numel())
    pos = torch.arange(n - rows, n, device="cuda")
    ref, vmax = dense64(t, c, q.view(rows, n_q, d), n_q, pos, window, sinks)
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    tol = (4e-5 + (2.0 ** -11 if dt != "f32" else 0.0)) * vmax + u * ref.abs()
    assert bool(((out.double().view_as(ref) - ref).abs() <= tol).all())
    # by the mean square: below the formats' own rounding by half again, f32 below 2e-6
    rel = float((out.double().view_as(ref) - ref).norm() / ref.norm())
    assert rel <= {"f32": 2e-6, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]


@pytest.mark.parametrize("window,sinks", [(5, 0), (64, 9), (300, 33)])
def test_window_at_other_head_sizes(window, sinks, ws):
    c = kvref.Cache(3, [90, 300, 1], 2, 16, 80, seed=window)
    check(*run(c, [3, 40, 1], "f32", 6, ws, window=window, sinks=sinks), "f32")


def test_two_streams_with_a_workspace_each(ws):
    import torch
    c = [kvref.Cache(1, [3000], 8, 64, 128, seed=40 + i) for i in range(2)]
    up = [upload(x) for x in c]
    q = [torch.randn(1, 32 * 128, device="cuda") for _ in range(2)]
    alone, both = ([torch.empty_like(x) for x in q] for _ in range(2))
    size = pq.pq_attn_ws_bytes(32, 8, 128)
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for i in range(2):
        pq.pq_attn(up[i][1], None, 1, "f32", q[i], 4096, 32, 0.088, 0, 0, alone[i], 4096, ws, ws.numel())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            pq.pq_attn(up[i][1], None, 1, "f32", q[i], 4096, 32, 0.088, 0, 0, both[i], 4096, spaces[i], size, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(alone[i], both[i])


def test_the_last_rows_of_a_token_split_over_row_tiles(ws):
    # 14 query heads per kv head: row tiles of 8, 16 and 256 rows end inside a token
    for dt, news in (("f32", [3, 1]), ("bf16", [2, 2]), ("f16", [41, 19])):
        c = kvref.Cache(2, [200, 133], 1, 32, 64, seed=51)
        check(*run(c, news, dt, 14, ws), dt)


def test_no_wait_ran_out():
    assert pq.pq_wait_timeouts() == 0
