"""The pool's entries and pq_attn_mod reject bad arguments on the host, before
any launch (fake addresses, never dereferenced)."""
import ctypes

import pytest

import quantized_weight_mat_gb300 as pq
from test_kv_refusals import built, cache  # noqa: F401
from test_kv_refusals import BUF, K, LEN, OUT, QKV, ROWS, TAB, V, WIDTH, WS

REFS, FROM, TO, TOK, NEW, ST = [(1 << 46) + (i << 36) for i in range(6)]
SLOPE, FIRST, PREFIX = [(1 << 47) + (i << 36) for i in range(3)]


def pool(**kw):
    a = dict(refs=REFS, table=TAB, len_=LEN, n_pages=64, page=64, n_seq=4, table_ld=16)
    a.update(kw)
    return pq.pq_kv_pool(*a.values())


def layer(i, **kw):
    at = (1 << 44) + (i << 40)
    return cache(k=at, v=at + (1 << 36), ks=at + (2 << 36), vs=at + (3 << 36), **kw)


def layers(n=2):
    return pq.pq_kv_layers([layer(i) for i in range(n)])


def fork(p, **kw):
    a = dict(n=2, from_=FROM, to=TO, tokens=TOK, ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    return pq.pq_kv_fork(p, *a.values(), stream=0, check=False)


def reserve(p, **kw):
    a = dict(layers=layers(), n_new=NEW, status=ST, ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    return pq.pq_kv_reserve(p, *a.values(), stream=0, check=False)


def free(p, **kw):
    a = dict(n=2, seq=FROM, begin=TO, end=TOK)
    a.update(kw)
    return pq.pq_kv_free(p, *a.values(), stream=0, check=False)


def compact(p, **kw):
    a = dict(layers=layers(), moved=NEW, n_used=ST, ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    return pq.pq_kv_compact(p, *a.values(), stream=0, check=False)


def attn(**kw):
    a = dict(row_start=0, n_rows=4, dt=0, q=QKV, ldq=WIDTH, n_q=32, scale=0.1, window=0, n_sink=0,
             mod=pq.pq_score_mod(30.0, SLOPE, FIRST, PREFIX), out=OUT, ldo=WIDTH, ws=WS, ws_bytes=1 << 30)
    a.update(kw)
    return pq.pq_attn_mod(cache(), *a.values(), stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(refs=0), pq.PQ_ERR_ARG), (dict(table=0), pq.PQ_ERR_ARG), (dict(len_=0), pq.PQ_ERR_ARG),
    (dict(n_pages=0), pq.PQ_ERR_ARG), (dict(n_seq=0), pq.PQ_ERR_ARG), (dict(table_ld=-1), pq.PQ_ERR_ARG),
    (dict(page=48), pq.PQ_ERR_LAYOUT), (dict(page=8), pq.PQ_ERR_LAYOUT),
    (dict(n_seq=65537), pq.PQ_ERR_SIZE), (dict(table_ld=1 << 25), pq.PQ_ERR_SIZE), (dict(n_pages=(1 << 28) + 1), pq.PQ_ERR_SIZE),
    (dict(n_seq=65536, table_ld=8192), pq.PQ_ERR_SIZE),
    (dict(refs=REFS + 4), pq.PQ_ERR_ALIGN), (dict(table=TAB + 2), pq.PQ_ERR_ALIGN), (dict(len_=LEN + 1), pq.PQ_ERR_ALIGN),
    (dict(refs=TAB + 64), pq.PQ_ERR_ARG), (dict(len_=TAB + 4), pq.PQ_ERR_ARG),
])
def test_pool_is_checked(kw, status):
    p = pool(**kw)
    assert fork(p) == free(p) == status
    if "n_pages" not in kw or kw["n_pages"] <= 0:
        assert reserve(p) == compact(p) == status
    overlaps = kw in (dict(refs=TAB + 64), dict(len_=TAB + 4))
    assert (pq.pq_kv_pool_ws_bytes(p) > 0) == overlaps


def test_null_pool():
    null = ctypes.POINTER(pq.KVPool)()
    assert pq.lib().pq_kv_free(null, 1, 0, 0, 0, 0) == pq.PQ_ERR_ARG
    assert pq.lib().pq_kv_pool_ws_bytes(null) == 0


@pytest.mark.parametrize("call", [fork, free])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), pq.PQ_ERR_ARG), (dict(n=5), pq.PQ_ERR_SIZE),
])
def test_lists_are_checked(call, kw, status):
    assert call(pool(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(from_=0), pq.PQ_ERR_ARG), (dict(to=0), pq.PQ_ERR_ARG), (dict(ws=0), pq.PQ_ERR_ARG),
    (dict(from_=FROM + 2), pq.PQ_ERR_ALIGN), (dict(tokens=TOK + 1), pq.PQ_ERR_ALIGN), (dict(ws=WS + 8), pq.PQ_ERR_ALIGN),
    (dict(ws_bytes=100), pq.PQ_ERR_WS),
    (dict(from_=TAB), pq.PQ_ERR_ARG), (dict(to=REFS + 8), pq.PQ_ERR_ARG), (dict(tokens=LEN), pq.PQ_ERR_ARG),
    (dict(tokens=WS + 4), pq.PQ_ERR_ARG), (dict(ws=TAB), pq.PQ_ERR_ARG),
])
def test_fork_is_checked(kw, status):
    assert fork(pool(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(seq=FROM + 1), pq.PQ_ERR_ALIGN), (dict(begin=LEN), pq.PQ_ERR_ARG), (dict(end=REFS), pq.PQ_ERR_ARG), (dict(seq=TAB + 8), pq.PQ_ERR_ARG),
])
def test_free_is_checked(kw, status):
    assert free(pool(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_new=0), pq.PQ_ERR_ARG), (dict(status=0), pq.PQ_ERR_ARG), (dict(ws=0), pq.PQ_ERR_ARG),
    (dict(n_new=NEW + 2), pq.PQ_ERR_ALIGN), (dict(status=ST + 1), pq.PQ_ERR_ALIGN), (dict(ws_bytes=64), pq.PQ_ERR_WS),
    (dict(status=NEW + 8), pq.PQ_ERR_ARG), (dict(n_new=LEN), pq.PQ_ERR_ARG), (dict(status=TAB), pq.PQ_ERR_ARG),
])
def test_reserve_is_checked(kw, status):
    assert reserve(pool(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_used=0), pq.PQ_ERR_ARG), (dict(n_used=ST + 2), pq.PQ_ERR_ALIGN), (dict(moved=NEW + 2), pq.PQ_ERR_ALIGN),
    (dict(ws_bytes=64), pq.PQ_ERR_WS), (dict(n_used=NEW + 16), pq.PQ_ERR_ARG), (dict(moved=REFS), pq.PQ_ERR_ARG),
    (dict(moved=WS), pq.PQ_ERR_ARG),
])
def test_compact_is_checked(kw, status):
    assert compact(pool(), **kw) == status


BAD_LAYERS = [
    ([layer(0), layer(1, n_pages=65)], pq.PQ_ERR_ARG),            # another pool's
    ([layer(0, page=32), layer(1)], pq.PQ_ERR_ARG),
    ([layer(0), layer(1, d=72)], pq.PQ_ERR_LAYOUT),
    ([layer(0), layer(1, n_kv=0)], pq.PQ_ERR_ARG),
    ([layer(0), cache(k=0)], pq.PQ_ERR_ARG),
    ([layer(0), layer(1), layer(0)], pq.PQ_ERR_ARG),              # the same layer twice
    ([layer(1), cache(k=(1 << 44) + (1 << 40) + 16)], pq.PQ_ERR_ARG),
    ([layer(0), cache(v=(1 << 44) + (2 << 36) + 16)], pq.PQ_ERR_ARG),      # codes over another's scales
    ([layer(0), cache(k=TAB + 16)], pq.PQ_ERR_ARG),
    ([layer(0), cache(k=WS + 4096)], pq.PQ_ERR_ARG),
    ([layer(0), cache(v=ST)], pq.PQ_ERR_ARG), ([layer(0), cache(v=NEW)], pq.PQ_ERR_ARG), ([layer(0), cache(v=REFS)], pq.PQ_ERR_ARG),
    ([layer(0), cache(k=K + 8)], pq.PQ_ERR_ALIGN),
]


@pytest.mark.parametrize("caches,status", BAD_LAYERS)
def test_layers_are_checked(caches, status):
    assert reserve(pool(), layers=pq.pq_kv_layers(caches)) == compact(pool(), layers=pq.pq_kv_layers(caches)) == status


def test_number_of_layers():
    L, p, one = pq.lib(), pool(), pq.pq_kv_layers([layer(0)])
    assert L.pq_kv_reserve(p, one, -1, NEW, ST, WS, 1 << 30, 0) == pq.PQ_ERR_ARG
    assert L.pq_kv_reserve(p, ctypes.POINTER(pq.KVCache)(), 1, NEW, ST, WS, 1 << 30, 0) == pq.PQ_ERR_ARG
    assert L.pq_kv_compact(p, one, 1025, 0, ST, WS, 1 << 30, 0) == pq.PQ_ERR_SIZE


@pytest.mark.parametrize("kw,status", [
    (dict(mod=pq.pq_score_mod(-1.0)), pq.PQ_ERR_ARG), (dict(mod=pq.pq_score_mod(float("nan"))), pq.PQ_ERR_ARG),
    (dict(mod=pq.pq_score_mod(float("inf"))), pq.PQ_ERR_ARG), (dict(mod=pq.pq_score_mod(1e-30)), pq.PQ_ERR_ARG),
    (dict(mod=pq.pq_score_mod(1e30)), pq.PQ_ERR_ARG),
    (dict(mod=pq.pq_score_mod(1.0, SLOPE + 2)), pq.PQ_ERR_ALIGN), (dict(mod=pq.pq_score_mod(0, 0, FIRST + 1)), pq.PQ_ERR_ALIGN),
    (dict(mod=pq.pq_score_mod(0, 0, 0, PREFIX + 3)), pq.PQ_ERR_ALIGN),
    (dict(mod=pq.pq_score_mod(0, OUT + 64)), pq.PQ_ERR_ARG), (dict(mod=pq.pq_score_mod(0, 0, WS + 64)), pq.PQ_ERR_ARG),
    (dict(mod=pq.pq_score_mod(0, 0, 0, OUT)), pq.PQ_ERR_ARG),
    (dict(ws_bytes=64), pq.PQ_ERR_WS), (dict(dt=3), pq.PQ_ERR_DTYPE), (dict(n_q=30), pq.PQ_ERR_LAYOUT), (dict(out=QKV), pq.PQ_ERR_ARG),
])
def test_attention_is_checked(kw, status):
    assert attn(**kw) == status


def test_workspace_sizes():
    assert pq.pq_attn_mod_ws_bytes(32, 8, 128, 100, 4) >= pq.pq_attn_ws_bytes(32, 8, 128)
    assert pq.pq_attn_mod_ws_bytes(30, 8, 128, 1, 1) == pq.pq_attn_mod_ws_bytes(32, 8, 128, -1, 1) == 0
    assert pq.pq_attn_mod_ws_bytes(32, 8, 128, 1, 0) == pq.pq_attn_mod_ws_bytes(32, 8, 128, 2 ** 31 - 1, 1) == 0
    assert pq.pq_kv_pool_ws_bytes(pool()) >= 64 + 28 * 64


def test_valid_arguments_reach_the_device_check():
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on a real GPU with fake pointers")
    p = pool()
    assert fork(p) == reserve(p) == free(p) == compact(p) == attn() == pq.PQ_ERR_DEVICE
    assert fork(p, tokens=0) == free(p, seq=0, begin=0, end=0) == pq.PQ_ERR_DEVICE
    assert fork(p, n=0, from_=0, to=0, tokens=0) == free(p, n=0, seq=0) == pq.PQ_ERR_DEVICE
    assert reserve(p, layers=None) == compact(p, layers=None, moved=0) == pq.PQ_ERR_DEVICE
    assert fork(p, from_=FROM, to=FROM) == pq.PQ_ERR_DEVICE                       # lists that are only read may be one
    # layers behind each other in one buffer per kind, in any order
    many = [cache(k=K + i * (64 * 8 * 64 * 128), v=V + i * (64 * 8 * 64 * 128), ks=BUF[2] + i * 2048, vs=BUF[3] + i * 2048)
            for i in (3, 0, 2, 1)]
    assert reserve(p, layers=pq.pq_kv_layers(many)) == pq.PQ_ERR_DEVICE
    assert attn(mod=None) == attn(mod=pq.pq_score_mod(), row_start=ROWS) == pq.PQ_ERR_DEVICE
    assert attn(mod=pq.pq_score_mod(0, SLOPE, FIRST, FIRST)) == pq.PQ_ERR_DEVICE


def test_the_status_text_names_the_workspaces():
    assert "pq_kv_pool_ws_bytes" in pq.pq_strerror(pq.PQ_ERR_WS)
