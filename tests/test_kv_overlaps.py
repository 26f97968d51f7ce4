"""What the paged-cache entries write overlaps nothing that they read: refused on
the host by columns where the row strides are equal (fake addresses, never
dereferenced: every call here is refused, or stops at the device check)."""
import pytest

import quantized_weight_mat_gb300 as pq
from test_kv_refusals import (COS, K, KO, KS, LEN, OUT, QKV, ROWS, SIN, TAB, V, VO, VS, WIDTH, WS, append, attn, built, cache,  # noqa: F401
                              gather)

ROW = 6144                  # a fused f32 row: 4096 of q, 1024 of k, 1024 of v
ARG, OK = pq.PQ_ERR_ARG, pq.PQ_ERR_DEVICE


@pytest.fixture
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on a real GPU with fake pointers")


def in_place(**kw):
    a = dict(q_out=QKV, ldq=ROW, ldqo=ROW, k=QKV + 4 * WIDTH, ldk=ROW, v=QKV + 4 * (WIDTH + 1024), ldv=ROW)
    a.update(kw)
    return append(cache(), **a)


@pytest.mark.parametrize("kw", [
    dict(k=QKV), dict(v=QKV), dict(k=QKV + 4 * (WIDTH - 16)), dict(v=QKV + 4 * 1024),
    dict(k=QKV + 4 * (WIDTH - 4)), dict(k=QKV + 4 * (ROW - 1020)),        # by four elements, at either side
    dict(k=QKV + 4 * ROW), dict(v=QKV - 4 * (ROW - 1024)),                 # another row's q
    dict(k=QKV, ldk=1024), dict(v=QKV + 4 * WIDTH, ldv=1024),              # strides of their own: by the whole span
])
def test_rotation_in_place_over_k_or_v_is_refused(kw):
    assert in_place(**kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(), dict(k=KO, ldk=1024, v=VO, ldv=1024), dict(k=QKV - 4 * 1024), dict(k=QKV + 4 * 4 * ROW, ldk=1024),
    dict(k=QKV + 4 * (4 * ROW)), dict(v=QKV - 4 * 4 * ROW),                # past the last row, before the first
])
def test_rotation_in_place_beside_k_and_v_is_taken(kw, no_gpu):
    assert in_place(**kw) == OK


@pytest.mark.parametrize("kw", [
    dict(q_out=QKV + 4 * ROW, ldq=2 * ROW, ldqo=2 * ROW),                                     # q_out beside q, in rows twice as long
    dict(q_out=QKV + 4 * (2 * ROW - WIDTH), ldq=2 * ROW, ldqo=2 * ROW),
    dict(q_out=QKV + 4 * ROW, ldq=2 * ROW, ldqo=2 * ROW, k=QKV + 4 * WIDTH, ldk=2 * ROW, v=QKV + 4 * (WIDTH + 1024), ldv=2 * ROW),
    dict(q_out=QKV + 4 * 3 * ROW + 4 * WIDTH, ldq=ROW, ldqo=ROW),                              # over no row's q, though between them
])
def test_other_columns_of_the_same_rows_are_taken(kw, no_gpu):
    assert append(cache(), **kw) == OK


@pytest.mark.parametrize("kw", [
    dict(q_out=QKV + 4 * (WIDTH - 4), ldq=2 * ROW, ldqo=2 * ROW), dict(q_out=QKV + 4 * (2 * ROW - WIDTH + 4), ldq=2 * ROW, ldqo=2 * ROW),
    dict(q_out=QKV + 4 * ROW, ldq=2 * ROW, ldqo=2 * ROW, v=QKV + 4 * (ROW + WIDTH - 4), ldv=2 * ROW),
    dict(q_out=QKV + 4 * ROW, ldq=2 * ROW, ldqo=2 * ROW, k=QKV + 4 * (ROW - 1020), ldk=2 * ROW),
    dict(q_out=QKV, ldq=ROW, ldqo=ROW + 4), dict(q_out=QKV + 4 * ROW, ldq=ROW, ldqo=ROW),       # the next row's q
])
def test_the_same_columns_are_refused(kw):
    assert append(cache(), **kw) == ARG


def test_attention_into_other_columns_is_taken(no_gpu):
    assert attn(cache(), out=QKV + 4 * WIDTH, ldq=2 * WIDTH, ldo=2 * WIDTH) == OK
    assert attn(cache(), out=QKV + 4 * ROW, ldq=2 * ROW, ldo=2 * ROW) == OK


@pytest.mark.parametrize("kw", [
    dict(out=QKV + 4 * (WIDTH - 4), ldq=2 * WIDTH, ldo=2 * WIDTH), dict(out=QKV + 4 * (WIDTH + 4), ldq=2 * WIDTH, ldo=2 * WIDTH),
    dict(out=QKV, ldq=2 * WIDTH, ldo=2 * WIDTH), dict(out=QKV + 4 * WIDTH, ldq=2 * WIDTH, ldo=WIDTH),
])
def test_attention_into_the_same_columns_is_refused(kw):
    assert attn(cache(), **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(row_start=OUT), dict(row_start=OUT + 4 * (4 * WIDTH - 4)), dict(row_start=K + 64), dict(row_start=VS + 4), dict(row_start=V),
    dict(rope_cos=OUT + 64), dict(rope_sin=OUT - 4 * 64 * 1023), dict(rope_sin=K), dict(rope_cos=VS),
    dict(q=K, q_out=OUT), dict(q=V + 4096, q_out=OUT), dict(q=VS, q_out=OUT),
])
def test_append_writes_nothing_that_it_reads(kw):
    assert append(cache(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(v=K), dict(v=K + 64 * 8 * 64 * 128 - 16), dict(vs=KS), dict(ks=V), dict(vs=K + 16), dict(table=K),
                                dict(len_=KS + 4), dict(table=VS)])
def test_append_writes_each_buffer_of_the_cache_once(kw):
    assert append(cache(**kw)) == ARG


def test_readers_may_share_buffers_of_the_cache(no_gpu):
    assert attn(cache(v=K, vs=KS)) == gather(cache(v=K, vs=KS)) == OK
    assert append(cache(), rope_sin=COS, k=KO, v=KO) == OK
    assert append(cache(), row_start=QKV) == OK


@pytest.mark.parametrize("kw", [dict(row_start=OUT), dict(row_start=WS + 1024), dict(row_start=OUT - 16), dict(ws=ROWS, row_start=ROWS + 64)])
def test_attention_writes_nothing_that_it_reads(kw):
    assert attn(cache(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(row_start=KO), dict(row_start=VO + 4 * 1024)])
def test_gather_writes_nothing_that_it_reads(kw):
    assert gather(cache(), **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(v_out=KO), dict(v_out=KO + 64), dict(v_out=KO + 4 * 3 * 1024), dict(v_out=KO - 4 * 1000),
    dict(ldk=2048, ldv=2048, v_out=KO + 4 * 1020), dict(ldk=2048, v_out=KO + 4 * 1024),
])
def test_gather_into_overlapping_rows_is_refused(kw):
    assert gather(cache(), **kw) == ARG


def test_gather_into_columns_of_one_buffer_is_taken(no_gpu):
    assert gather(cache(), ldk=2048, ldv=2048, v_out=KO + 4 * 1024) == OK
    assert gather(cache(), v_out=KO + 4 * 4 * 1024) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("news", [None, [40, 3, 70]])
def test_columns_of_one_buffer_as_buffers_of_their_own(dt, news, cuda_ok):
    # [q | k | v | rotated q | attention] in each row against the same calls on buffers of their own
    import numpy as np
    import torch

    import kvref
    from test_gpu_kv_cache import tables, tdt, upload
    n_q, n_kv, d = 4, 2, 64
    lens = [100, 17, 70]
    rows = 3 if news is None else sum(news)
    rs = None if news is None else torch.tensor([0] + np.cumsum(news).tolist(), dtype=torch.int32, device="cuda")
    w, kw = n_q * d, n_kv * d
    full = 3 * w + 2 * kw
    x = torch.randn(rows, full, device="cuda").to(tdt(dt))
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(100, d))
    ws = torch.empty(pq.pq_attn_ws_bytes(n_q, n_kv, d), dtype=torch.uint8, device="cuda")
    got = []
    for apart in (False, True):
        t, h = upload(kvref.Cache(3, lens, n_kv, 16, d, seed=3))
        b = x.clone()
        q, k, v = b[:, :w], b[:, w:], b[:, w + kw:]
        turned, out = (torch.empty(rows, w, dtype=b.dtype, device="cuda") for _ in range(2)) if apart else (b[:, w + 2 * kw:], b[:, 2 * w + 2 * kw:])
        ld = w if apart else full
        pq.pq_kv_append(h, rs, rows, dt, k, full, v, full, q, full, n_q, turned, ld, cos, sin, 100, d, "half")
        pq.pq_attn(h, rs, rows, dt, turned, ld, n_q, d ** -0.5, 0, 0, out, ld, ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(b[:, :w + 2 * kw], x[:, :w + 2 * kw])
        got.append([turned[:, :w].contiguous(), out[:, :w].contiguous()] + [t[n] for n in ("k", "v", "ks", "vs")])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))
