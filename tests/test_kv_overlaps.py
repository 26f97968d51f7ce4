"""What the paged-cache entries write overlaps nothing that they read: refused on
the host by columns where the row strides are equal (fake addresses, never
dereferenced: every call here is refused, or stops at the device check)."""
import pytest

import quantized_weight_mat_gb300 as pq
from test_kv_refusals import KO, OUT, QKV, VO, WIDTH, append, built, cache  # noqa: F401

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
