"""Append to and gather from the paged 8-bit cache on the GPU: codes, scales
and values bit for bit as pq.h states them (tests/kvref.py), and against the
rotation and quantization in 64 bits within half a step."""
import numpy as np
import pytest

import kvref
import quantized_weight_mat_gb300 as pq

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


def tdt(dt):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt]


def upload(c):
    import torch
    t = {n: torch.from_numpy(getattr(c, n).copy()).cuda() for n in ("k", "v", "ks", "vs", "table", "len")}
    h = pq.pq_kv_cache(t["k"], t["v"], t["ks"], t["vs"], t["table"], t["len"], c.n_pages, c.n_kv, c.page, c.d, c.n_seq,
                       c.table_ld)
    return t, h


def tables(n_pos, rot, seed=3):
    rng = np.random.default_rng(seed)
    a = rng.uniform(-np.pi, np.pi, (n_pos, max(rot // 2, 1)))
    return np.cos(a).astype(F32), np.sin(a).astype(F32)


def run_append(c, news, dt, rot, mode, n_q, seed, pad=8, in_place=False, make=None, n_pos=None, rows_given=True):
    """Append on the GPU and by the reference; checks everything that is written."""
    import torch
    row_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n_rows = int(row_start[-1])
    rng = np.random.default_rng(seed)
    wide = (n_q + 2 * c.n_kv) * c.d + pad
    qkv = torch.from_numpy(rng.normal(0, 1, (n_rows, wide)).astype(F32))
    if make:
        make(qkv, n_q * c.d, c)
    qkv = qkv.to(tdt(dt)).cuda()
    f = qkv.float().cpu().numpy()
    cos, sin = tables(n_pos or int(max(c.len.max(), 1)), rot)
    tc, ts = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    t, h = upload(c)
    rs = torch.from_numpy(row_start).cuda() if rows_given else None
    k, v = qkv[:, n_q * c.d:], qkv[:, (n_q + c.n_kv) * c.d:]
    guard = torch.full((n_rows + 1, n_q * c.d + 16), 77.0, dtype=tdt(dt), device="cuda")
    q_out, ldo = (qkv, wide) if in_place else (guard, n_q * c.d + 16)
    pq.pq_kv_append(h, rs, n_rows, dt, k, wide, v, wide, qkv, wide, n_q, q_out, ldo, tc, ts, cos.shape[0], rot, mode)
    torch.cuda.synchronize()
    kn = f[:, n_q * c.d:(n_q + c.n_kv) * c.d].reshape(n_rows, c.n_kv, c.d)
    vn = f[:, (n_q + c.n_kv) * c.d:(n_q + 2 * c.n_kv) * c.d].reshape(n_rows, c.n_kv, c.d)
    rs_np = row_start if rows_given else None
    kvref.append(c, rs_np, kn, vn, cos, sin, rot, mode)
    for name in ("ks", "vs"):
        assert np.array_equal(t[name].cpu().numpy(), getattr(c, name), equal_nan=True), name
    for name in ("k", "v"):
        assert np.array_equal(t[name].cpu().numpy(), getattr(c, name)), name
    # the rotated queries
    want = np.empty((n_rows, n_q, c.d), F32)
    for r, (_, pos) in enumerate(kvref.places(c, rs_np, n_rows)):
        x = f[r, :n_q * c.d].reshape(n_q, c.d)
        p = max(pos, 0)
        nan = np.full(max(rot // 2, 1), np.nan, F32)
        want[r] = kvref.rotate(x, cos[p] if p < len(cos) else nan, sin[p] if p < len(cos) else nan, rot, mode) if rot else x
    want = torch.from_numpy(want.reshape(n_rows, -1)).to(tdt(dt))
    got = q_out[:n_rows, :n_q * c.d].cpu()
    assert torch.equal(torch.nan_to_num(got.float(), nan=1e30), torch.nan_to_num(want.float(), nan=1e30))
    if in_place:      # the columns beside q stay as they were
        assert np.array_equal(qkv[:, n_q * c.d:].float().cpu().numpy(), f[:, n_q * c.d:], equal_nan=True)
    else:
        assert torch.all(guard[n_rows] == 77.0) and torch.all(guard[:, n_q * c.d:] == 77.0)
    # and back
    ko = torch.full((n_rows + 1, c.n_kv * c.d + 8), 55.0, dtype=tdt(dt), device="cuda")
    vo = torch.full_like(ko, 55.0)
    pq.pq_kv_gather(h, rs, n_rows, dt, ko, c.n_kv * c.d + 8, vo, c.n_kv * c.d + 8)
    torch.cuda.synchronize()
    for o, want in zip((ko, vo), kvref.gather(c, rs_np, n_rows)):
        w = torch.from_numpy(want.reshape(n_rows, -1)).to(tdt(dt)).float().numpy()
        assert np.array_equal(o[:n_rows, :c.n_kv * c.d].float().cpu().numpy(), w, equal_nan=True)
        assert torch.all(o[n_rows] == 55.0) and torch.all(o[:, c.n_kv * c.d:] == 55.0)
    return t, h, f


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("mode,rot,d", [("half", 128, 128), ("pair", 128, 128), ("half", 32, 64), ("pair", 16, 64), ("half", 0, 64),
                                        ("half", 80, 80), ("pair", 256, 256)])
def test_append_ragged(dt, page, mode, rot, d):
    # starts inside a page, at its first token, over several pages, nothing, an idle slot
    lens = [1, page, page + 1, 3 * page - 1, 0, 2 * page + 5, 7]
    news = [1, page, 1, 2 * page + 3, 0, page + 5, 7]
    c = kvref.Cache(len(lens), lens, 2, page, d, seed=page + d)
    run_append(c, news, dt, rot, mode, n_q=4, seed=11)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n_seq", [1, 5, 130])
def test_append_one_token_each(dt, n_seq):
    lens = [0 if i % 7 == 3 else 1 + (37 * i) % 200 for i in range(n_seq)]
    c = kvref.Cache(n_seq, lens, 8, 32, 128, seed=n_seq)
    run_append(c, [1] * n_seq, dt, 128, "half", n_q=32, seed=5, rows_given=False)


def test_many_sequences_with_rows_given():
    n_seq = 300                                    # more than one pass of the search over sequences
    news = [i % 4 for i in range(n_seq)]
    lens = [m + (13 * i) % 50 for i, m in enumerate(news)]
    c = kvref.Cache(n_seq, lens, 1, 16, 64, seed=8)
    run_append(c, news, "f16", 64, "half", n_q=2, seed=6)


def test_in_place_rotation_beside_k_and_v():
    c = kvref.Cache(2, [70, 33], 2, 32, 128, seed=4)
    run_append(c, [40, 3], "f32", 64, "half", n_q=8, seed=9, in_place=True)
    c = kvref.Cache(2, [70, 33], 2, 32, 128, seed=4)
    run_append(c, [40, 3], "f16", 128, "pair", n_q=8, seed=9, in_place=True)


def test_growing_scale_rescales_older_tokens():
    lens, page = [20], 32
    c = kvref.Cache(1, lens, 1, page, 64, seed=2)
    before, s0 = c.k.copy(), c.ks.copy()

    def big(qkv, at, c):
        qkv[:, at:] *= 40.0
    t, _, _ = run_append(c, [1], "f32", 0, "half", n_q=1, seed=3, make=big)
    pg = c.table[0, 0]
    assert c.ks[pg, 0] > s0[pg, 0]
    # in 64 bits: each older value moves by at most half a step of the new scale
    was = before[pg, 0, :19].astype(np.float64) * float(s0[pg, 0])
    now = t["k"].cpu().numpy()[pg, 0, :19].astype(np.float64) * float(c.ks[pg, 0])
    assert np.abs(was - now).max() <= 0.5 * float(c.ks[pg, 0]) * (1 + 1e-5)


def test_quantization_error_in_64_bits():
    # rotation and quantization within half a step, plus the rotation's f32 rounding (3 roundings of values below 8)
    page, d, n = 64, 128, 150
    c = kvref.Cache(1, [n], 2, page, d, seed=12)
    t, _, f = run_append(c, [n], "f32", d, "half", n_q=2, seed=13)
    cos, sin = (x.astype(np.float64) for x in tables(n, d))
    k = f[:, 2 * d:4 * d].reshape(n, 2, d).astype(np.float64)
    a, b = k[..., :64], k[..., 64:]
    turned = np.concatenate([a * cos[:, None] - b * sin[:, None], a * sin[:, None] + b * cos[:, None]], -1)
    codes = t["k"].cpu().numpy()
    for pos in range(n):
        pg = c.table[0, pos // page]
        step = c.ks[pg].astype(np.float64)[:, None]
        err = np.abs(codes[pg, :, pos % page] * step - turned[pos])
        assert (err <= 0.5 * step * (1 + 1e-5) + 3 * 8 * 2.0 ** -24).all()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_non_finite_values_poison_their_page_only(bad):
    lens, page = [40, 40], 16

    def put(qkv, at, c):
        qkv[3, at + 5] = bad
    c = kvref.Cache(2, lens, 1, page, 64, seed=7)
    t, h, _ = run_append(c, [40, 40], "f32", 0, "half", n_q=1, seed=1, make=put)
    assert np.isnan(c.ks[c.table[0, 0], 0]) and np.isfinite(c.ks[c.table[0, 1:], 0]).all()
    assert np.isfinite(c.vs[c.table[:, :3], 0]).all() and np.isfinite(c.ks[c.table[1], 0]).all()
    # writing the page from its first token again clears it
    c.len[:] = [16, 40]
    run_append(c, [16, 1], "f32", 0, "half", n_q=1, seed=2)
    assert np.isfinite(c.ks[c.table[0, 0], 0])


def test_zero_and_tiny_values():
    def tiny(qkv, at, c):
        qkv[:16, at:] = 0.0
        qkv[16:, at:] = 1e-39
    c = kvref.Cache(1, [32], 1, 16, 64, seed=7)
    run_append(c, [32], "f32", 0, "half", n_q=1, seed=1, make=tiny)
    assert (c.ks[c.table[0]] == 0).all()


def test_positions_outside_the_cache_are_left_out():
    # missing pages, a table too short for the length, more rows than tokens, positions past the rotation's table
    c = kvref.Cache(3, [70, 90, 5], 2, 16, 64, seed=21, table_ld=4)
    c.table[0, 2] = -1
    c.table[1, 0] = c.n_pages
    c.table[1, 1] = -(1 << 31)
    run_append(c, [50, 90, 9], "f32", 64, "half", n_q=2, seed=2, n_pos=60)


def test_repeating_an_append_changes_nothing():
    import torch
    c = kvref.Cache(1, [29], 2, 16, 64, seed=31)
    t, h, f = run_append(c, [11], "f32", 0, "half", n_q=2, seed=3)
    first = [t[n].clone() for n in ("k", "v", "ks", "vs")]
    x = torch.from_numpy(f).cuda()
    rs = torch.tensor([0, 11], dtype=torch.int32, device="cuda")
    pq.pq_kv_append(h, rs, 11, "f32", x[:, 128:], x.shape[1], x[:, 256:], x.shape[1])
    torch.cuda.synchronize()
    for a, n in zip(first, ("k", "v", "ks", "vs")):
        assert torch.equal(a.view(torch.uint8), t[n].view(torch.uint8))


def test_no_rows_is_nothing_to_do():
    import torch
    c = kvref.Cache(2, [5, 6], 1, 16, 64, seed=1)
    t, h = upload(c)
    x = torch.zeros(16, 192, device="cuda")
    rs = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert pq.pq_kv_append(h, rs, 0, "f32", x[:, 64:], 192, x[:, 128:], 192) == 0
    assert pq.pq_kv_gather(h, rs, 0, "f32", x, 64, x, 64) == 0
    torch.cuda.synchronize()
    assert np.array_equal(t["k"].cpu().numpy(), c.k)


def test_offsets_past_32_bits_and_another_stream():
    import torch
    n_kv, page, d = 8, 64, 128
    n_pages = 2 ** 31 // (n_kv * page * d) + 64         # the last pages lie past 2^31 bytes
    k = torch.zeros(n_pages, n_kv, page, d, dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros(n_pages, n_kv, device="cuda")
    vs = torch.zeros_like(ks)
    table = torch.tensor([[n_pages - 1, 0]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([70], dtype=torch.int32, device="cuda")
    rs = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    x = torch.randn(70, 2 * n_kv * d, device="cuda")
    h = pq.pq_kv_cache(k, v, ks, vs, table, ln, n_pages, n_kv, page, d, 1, 2)
    out = torch.empty(2, 70, n_kv * d, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pq.pq_kv_append(h, rs, 70, "f32", x, 2 * n_kv * d, x[:, n_kv * d:], 2 * n_kv * d, stream=side)
    pq.pq_kv_gather(h, rs, 70, "f32", out[0], n_kv * d, out[1], n_kv * d, stream=side)
    side.synchronize()
    step = torch.cat([ks[n_pages - 1].repeat(64, 1), ks[0].repeat(6, 1)]).repeat_interleave(d, 1)
    assert torch.all((out[0] - x[:, :n_kv * d]).abs() <= 0.5 * step * (1 + 1e-5))
    assert int(k[n_pages - 1].abs().max()) == 127 and int(k[1:n_pages - 1].abs().max()) == 0
