"""Calls of the paged-cache entries at the edges of their arguments: no rows, and
no queries to rotate."""
import pytest

import quantized_weight_mat_gb300 as pq
from test_kv_refusals import ROWS, append, attn, built, cache, gather  # noqa: F401


def test_no_rows_need_no_buffers():
    # an empty tensor has no address; nothing is read, written or launched
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake table would pass the device check")
    for rs in (ROWS, ROWS + 64):
        assert attn(cache(), n_rows=0, row_start=rs, q=0, out=0) == pq.PQ_ERR_DEVICE
        assert append(cache(), n_rows=0, row_start=rs, k=0, v=0, q=0, q_out=0) == pq.PQ_ERR_DEVICE
        assert gather(cache(), n_rows=0, row_start=rs, k_out=0, v_out=0) == pq.PQ_ERR_DEVICE


@pytest.mark.parametrize("n_rows", [1, 4])
def test_rows_need_their_buffers(n_rows):
    kw = dict(n_rows=n_rows, row_start=ROWS)
    assert attn(cache(), q=0, **kw) == attn(cache(), out=0, **kw) == pq.PQ_ERR_ARG
    assert append(cache(), k=0, **kw) == append(cache(), v=0, **kw) == append(cache(), q_out=0, **kw) == pq.PQ_ERR_ARG
    assert gather(cache(), k_out=0, **kw) == gather(cache(), v_out=0, **kw) == pq.PQ_ERR_ARG


@pytest.mark.gpu
def test_no_rows_from_empty_tensors(cuda_ok):
    import torch

    import kvref
    from test_gpu_kv_cache import upload
    c = kvref.Cache(2, [5, 6], 1, 16, 64, seed=1)
    t, h = upload(c)
    before = [t[n].clone() for n in ("k", "v", "ks", "vs")]
    rs = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 64, device="cuda")
    ws = torch.empty(pq.pq_attn_ws_bytes(1, 1, 64), dtype=torch.uint8, device="cuda")
    assert pq.pq_kv_append(h, rs, 0, "f32", none, 64, none, 64, none, 64, 1, none, 64) == 0
    assert pq.pq_kv_gather(h, rs, 0, "f32", none, 64, none, 64) == 0
    assert pq.pq_attn(h, rs, 0, "f32", none, 64, 1, 1.0, 0, 0, none, 64, ws, ws.numel()) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), t[n].view(torch.uint8)) for a, n in zip(before, ("k", "v", "ks", "vs")))


@pytest.mark.gpu
@pytest.mark.parametrize("rows_given", [False, True])
@pytest.mark.parametrize("n_q", [0, 7, 1 << 30, -5])
def test_without_q_its_head_count_does_not_matter(n_q, rows_given, cuda_ok):
    import torch

    import kvref
    from test_gpu_kv_cache import upload
    c = kvref.Cache(2, [5, 36], 2, 16, 64, seed=1)
    rs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda") if rows_given else None
    x = torch.randn(2, 256, device="cuda")
    got = []
    for n in (0, n_q):
        t, h = upload(c)
        pq.pq_kv_append(h, rs, 2, "f32", x, 256, x[:, 128:], 256, n_q=n)
        torch.cuda.synchronize()
        got.append([t[k] for k in ("k", "v", "ks", "vs")])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))
