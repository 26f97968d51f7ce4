"""The paged-cache and attention entries reject bad arguments on the host,
before any launch (fake addresses, never dereferenced)."""
import ctypes

import pytest

import quantized_weight_mat_gb300 as pq

A = 1 << 40          # 16-byte aligned fake addresses, far apart
BUF = [A + (i << 36) for i in range(16)]
K, V, KS, VS, TAB, LEN, QKV, OUT, WS, COS, SIN, KO, VO, ROWS = BUF[:14]
WIDTH = 32 * 128


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_mat_gb300 import build
    build.build()


def cache(**kw):
    a = dict(k=K, v=V, ks=KS, vs=VS, table=TAB, len_=LEN, n_pages=64, n_kv=8, page=64, d=128, n_seq=4, table_ld=16)
    a.update(kw)
    return pq.pq_kv_cache(a["k"], a["v"], a["ks"], a["vs"], a["table"], a["len_"], a["n_pages"], a["n_kv"], a["page"],
                          a["d"], a["n_seq"], a["table_ld"])


def attn(c, **kw):
    a = dict(row_start=0, n_rows=4, dt=0, q=QKV, ldq=WIDTH, n_q=32, scale=0.1, window=0, n_sink=0, out=OUT, ldo=WIDTH,
             ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    return pq.pq_attn(c, *a.values(), stream=0, check=False)


def append(c, **kw):
    a = dict(row_start=0, n_rows=4, dt=0, k=KO, ldk=1024, v=VO, ldv=1024, q=QKV, ldq=WIDTH, n_q=32, q_out=OUT, ldqo=WIDTH,
             rope_cos=COS, rope_sin=SIN, n_pos=1024, rot=128, rope_mode=0)
    a.update(kw)
    return pq.pq_kv_append(c, *a.values(), stream=0, check=False)


def gather(c, **kw):
    a = dict(row_start=0, n_rows=4, dt=0, k_out=KO, ldk=1024, v_out=VO, ldv=1024)
    a.update(kw)
    return pq.pq_kv_gather(c, *a.values(), stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), pq.PQ_ERR_ARG), (dict(vs=0), pq.PQ_ERR_ARG), (dict(table=0), pq.PQ_ERR_ARG), (dict(len_=0), pq.PQ_ERR_ARG),
    (dict(n_pages=0), pq.PQ_ERR_ARG), (dict(n_kv=-1), pq.PQ_ERR_ARG), (dict(n_seq=0), pq.PQ_ERR_ARG),
    (dict(table_ld=0), pq.PQ_ERR_ARG),
    (dict(n_seq=5), pq.PQ_ERR_ARG),                                # one row per sequence, but 4 rows
    (dict(page=48), pq.PQ_ERR_LAYOUT), (dict(page=256), pq.PQ_ERR_LAYOUT),
    (dict(d=72), pq.PQ_ERR_LAYOUT), (dict(d=272), pq.PQ_ERR_LAYOUT), (dict(d=0), pq.PQ_ERR_LAYOUT),
    (dict(table_ld=1 << 25), pq.PQ_ERR_SIZE), (dict(n_pages=1 << 30), pq.PQ_ERR_SIZE),
    (dict(k=K + 8), pq.PQ_ERR_ALIGN), (dict(ks=KS + 2), pq.PQ_ERR_ALIGN), (dict(table=TAB + 1), pq.PQ_ERR_ALIGN),
])
def test_cache_is_checked(kw, status):
    c = cache(**kw)
    n = 4
    assert attn(c, n_rows=n) == status
    assert append(c, n_rows=n) == status
    assert gather(c, n_rows=n) == status


def test_null_handle():
    L = pq.lib()
    assert L.pq_kv_gather(ctypes.POINTER(pq.KVCache)(), 0, 4, 0, KO, 1024, VO, 1024, 0) == pq.PQ_ERR_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), pq.PQ_ERR_DTYPE), (dict(dt=-1), pq.PQ_ERR_DTYPE),
    (dict(n_rows=-1), pq.PQ_ERR_ARG), (dict(q=0), pq.PQ_ERR_ARG), (dict(out=0), pq.PQ_ERR_ARG), (dict(ws=0), pq.PQ_ERR_ARG),
    (dict(n_q=0), pq.PQ_ERR_ARG), (dict(n_q=30), pq.PQ_ERR_LAYOUT),
    (dict(ldq=WIDTH - 4), pq.PQ_ERR_ARG), (dict(ldq=WIDTH + 2), pq.PQ_ERR_ALIGN), (dict(q=QKV + 4), pq.PQ_ERR_ALIGN),
    (dict(out=OUT + 8), pq.PQ_ERR_ALIGN), (dict(ws=WS + 4), pq.PQ_ERR_ALIGN), (dict(ldo=1 << 60), pq.PQ_ERR_SIZE),
    (dict(window=-1), pq.PQ_ERR_ARG), (dict(n_sink=-1), pq.PQ_ERR_ARG),
    (dict(scale=float("nan")), pq.PQ_ERR_ARG), (dict(scale=float("inf")), pq.PQ_ERR_ARG),
    (dict(ws_bytes=8), pq.PQ_ERR_WS),
    (dict(out=QKV), pq.PQ_ERR_ARG), (dict(out=K + 1024), pq.PQ_ERR_ARG), (dict(ws=OUT + 64), pq.PQ_ERR_ARG),
])
def test_attention_is_checked(kw, status):
    assert attn(cache(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), pq.PQ_ERR_DTYPE),
    (dict(k=0), pq.PQ_ERR_ARG), (dict(v=0), pq.PQ_ERR_ARG), (dict(ldk=1020), pq.PQ_ERR_ARG), (dict(ldv=1026), pq.PQ_ERR_ALIGN),
    (dict(q=0), pq.PQ_ERR_ARG), (dict(q_out=0), pq.PQ_ERR_ARG),      # both or neither
    (dict(n_q=12), pq.PQ_ERR_LAYOUT), (dict(rot=24), pq.PQ_ERR_LAYOUT), (dict(rot=144), pq.PQ_ERR_LAYOUT),
    (dict(rot=-16), pq.PQ_ERR_LAYOUT), (dict(rope_mode=2), pq.PQ_ERR_ARG), (dict(rope_cos=0), pq.PQ_ERR_ARG),
    (dict(n_pos=0), pq.PQ_ERR_ARG), (dict(rope_sin=SIN + 4), pq.PQ_ERR_ALIGN),
    (dict(q_out=QKV + 64), pq.PQ_ERR_ARG), (dict(q_out=KO), pq.PQ_ERR_ARG), (dict(k=K), pq.PQ_ERR_ARG),
])
def test_append_is_checked(kw, status):
    assert append(cache(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=9), pq.PQ_ERR_DTYPE), (dict(k_out=0), pq.PQ_ERR_ARG), (dict(ldv=8), pq.PQ_ERR_ARG),
    (dict(k_out=KO + 4), pq.PQ_ERR_ALIGN), (dict(v_out=V), pq.PQ_ERR_ARG),
])
def test_gather_is_checked(kw, status):
    assert gather(cache(), **kw) == status


def test_valid_arguments_reach_the_device_check():
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on a real GPU with fake pointers")
    assert attn(cache()) == append(cache()) == gather(cache()) == pq.PQ_ERR_DEVICE
    # q may be rotated in place beside k and v; no rotation needs no tables
    assert append(cache(), q_out=QKV, k=QKV + 4 * WIDTH, ldk=6144, ldq=6144, ldqo=6144) == pq.PQ_ERR_DEVICE
    assert append(cache(), rot=0, rope_cos=0, rope_sin=0, n_pos=0, q=0, q_out=0, n_q=0) == pq.PQ_ERR_DEVICE


def test_workspace_size():
    assert pq.pq_attn_ws_bytes(32, 8, 128) > 0
    assert pq.pq_attn_ws_bytes(30, 8, 128) == pq.pq_attn_ws_bytes(32, 8, 100) == pq.pq_attn_ws_bytes(0, 8, 128) == 0


def test_strerror_names_the_new_codes():
    for st in (pq.PQ_ERR_DTYPE, pq.PQ_ERR_LAYOUT, pq.PQ_ERR_WS):
        assert pq.pq_strerror(st) != "unknown status"
