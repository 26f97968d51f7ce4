"""pq_attn_mod at the ends of what it takes: caps far above the scores, slopes whose bias overflows f32 or that are no numbers.

Bounds as in test_gpu_attn.py: 4e-5 for the scores (times `wide`, how much larger than usual they are), 2^-11 for the weights
of 16-bit rows, the output's own rounding.  The cap's error is 2^-21 of a capped score (below 16 * wide times log2 e), or
of the cap in calls of 16-bit rows with a cap of at most 256: never of a larger cap.
"""
import numpy as np
import pytest

import kvref
import modref
import quantized_weight_mat_gb300 as pq
from test_gpu_attn import DTS, ws  # noqa: F401
from test_gpu_attn_mod import LOG2E
from test_gpu_kv_cache import tdt, upload

pytestmark = pytest.mark.gpu
HEADS = [(8, 2, 128), (8, 2, 64), (4, 2, 80)]
NEWS = [None, [3], [40], [300]]          # one row; one and two blocks of rows; the prompt kernel


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def attend(c, news, dt, n_q, ws, qmul=1.0, cap=0.0, slope=None, first=None, prefix=None, window=0, sinks=0):  # noqa: F811
    """(out, 64-bit out, largest visible |v|)"""
    import torch
    row_start = None if news is None else np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n, w, scale = 1 if news is None else int(row_start[-1]), n_q * c.d, c.d ** -0.5
    q = torch.from_numpy(np.random.default_rng(7).normal(0, qmul, (n, w)).astype(np.float32)).to(tdt(dt)).cuda()
    _, h = upload(c)
    out = torch.full((n, w), 99.0, dtype=tdt(dt), device="cuda")
    size = pq.pq_attn_mod_ws_bytes(n_q, c.n_kv, c.d, n, 1)
    pq.pq_attn_mod(h, dev(row_start), n, dt, q, w, n_q, scale, window, sinks, pq.pq_score_mod(cap, dev(slope), dev(first), dev(prefix)),
                   out, w, ws, size)
    torch.cuda.synchronize()
    qf = q.float().cpu().numpy().reshape(n, n_q, c.d)
    ref, vmax = modref.attention(c, row_start, qf, n_q, scale, window, sinks, cap, slope, first, prefix)
    return out.float().cpu().numpy().reshape(n, n_q, c.d), ref, vmax


def check(got, ref, vmax, dt, off=0.0, wide=1.0):
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    tol = (4e-5 * wide + 2 * 0.6932 * off + (2.0 ** -11 if dt != "f32" else 0.0)) * vmax[..., None] + u * np.abs(ref) + 1e-30
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound"


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("cap", [257.0, 1e3, 1e4, 1e5, 1e6, 1e9, 2.0 ** 40, 2.0 ** 60])
def test_caps_far_above_the_scores(dt, heads, news, cap, ws):  # noqa: F811
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 32, d, seed=21)
    check(*attend(c, news, dt, n_q, ws, cap=cap), dt, off=2.0 ** -21 * LOG2E * 16)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("cap", [256.0, 300.0])
def test_scores_that_a_large_cap_bends(dt, heads, news, cap, ws):  # noqa: F811
    # scores of up to some 300 on both sides of the cap where the form changes
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 32, d, seed=22)
    check(*attend(c, news, dt, n_q, ws, cap=cap, qmul=60.0), dt, off=2.0 ** -21 * LOG2E * max(16 * 60, cap), wide=60.0)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("news", NEWS)
def test_large_caps_beside_biases_and_views(dt, heads, news, ws):  # noqa: F811
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 16, d, seed=23)
    c.table[0, 7] = -1
    n = 1 if news is None else news[0]
    off = 2.0 ** -21 * LOG2E * 16
    bias = 3 * 2.0 ** -24 * LOG2E * 64
    check(*attend(c, news, dt, n_q, ws, cap=1e6, slope=modref.slopes(n_q)), dt, off=off + bias)
    first = np.random.default_rng(23).integers(0, 650, n).astype(np.int32)
    check(*attend(c, news, dt, n_q, ws, cap=1e6, first=first, prefix=np.full(n, 640, np.int32), window=90, sinks=20), dt, off=off)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("news", NEWS)
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_slopes_whose_bias_overflows(dt, heads, news, cap, ws):  # noqa: F811
    # the nearest token alone, or with a negative slope the farthest: distances go to 3000, 1.2e35 * 3000 is past f32
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [3000], n_kv, 32, d, seed=24)
    n = 1 if news is None else news[0]
    slope = np.array([1.2e35, -1.2e35, 3e38, 1.0, 1e36, -3e38, 0.0, -1e36], np.float32)[:n_q]
    off = (2.0 ** -21 * LOG2E * (16 if dt == "f32" else max(cap, 16)) if cap else 0.0) + 3 * 2.0 ** -24 * LOG2E * 64
    check(*attend(c, news, dt, n_q, ws, cap=cap, slope=slope), dt, off=off)
    # rows that see nothing but what lies ahead of them, or nothing at all
    pos = np.arange(3000 - n, 3000)
    args = dict(first=(pos + 2).astype(np.int32), prefix=np.full(n, 3000, np.int32))
    check(*attend(c, news, dt, n_q, ws, cap=cap, slope=slope, **args), dt, off=off + 3 * 2.0 ** -24 * LOG2E * 2 * n)
    # and the page of the nearest ones is not there
    c.table[0, -4:] = -1
    check(*attend(c, news, dt, n_q, ws, cap=cap, slope=slope), dt, off=off + 3 * 2.0 ** -24 * LOG2E * 128)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("news", NEWS)
def test_a_slope_that_is_no_number_spoils_its_own_head(dt, heads, news, ws):  # noqa: F811
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [700], n_kv, 32, d, seed=25)
    slope = np.array([1.0, np.inf, np.nan, -np.inf, 0.25, 0.0, -0.01, 0.5], np.float32)[:n_q]
    sane = np.where(np.isfinite(slope), slope, 0.0).astype(np.float32)
    n = 1 if news is None else news[0]
    for views in ({}, dict(first=(np.arange(700 - n, 700) + 2).astype(np.int32), prefix=np.full(n, 700, np.int32))):
        got, _, _ = attend(c, news, dt, n_q, ws, slope=slope, **views)
        _, ref, vmax = attend(c, news, dt, n_q, ws, slope=sane, **views)
        sees = vmax > 0
        bad = ~np.isfinite(slope)
        assert np.isnan(got[:, bad][sees[:, bad]]).all()
        assert (got[~sees] == 0).all()
        check(got[:, ~bad], ref[:, ~bad], vmax[:, ~bad], dt, off=3 * 2.0 ** -24 * LOG2E * (64 + 7))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("starts", [[0, 200, 50, 300], [300, 0, 300, 300], [0, 9, 3, 12], [0, 400, -5, 300]])
def test_rows_that_fall(dt, d, starts, ws):  # noqa: F811
    # sequences share rows, against the rule: nothing is written, and the next call is as ever
    import torch
    c = kvref.Cache(3, [900, 700, 800], 2, 32, d, seed=26)
    _, h = upload(c)
    n, w = 300, 8 * d
    q = torch.randn(n, w, device="cuda").to(tdt(dt))
    first = dev(np.random.default_rng(26).integers(0, 900, n).astype(np.int32))
    size = pq.pq_attn_mod_ws_bytes(8, 2, d, n, 3)
    outs = []
    for rows in ([0, 100, 200, 300], starts, [0, 100, 200, 300]):
        out = torch.full((n, w), 99.0, dtype=q.dtype, device="cuda")
        pq.pq_attn_mod(h, dev(np.array(rows, np.int32)), n, dt, q, w, 8, 0.1, 0, 0, pq.pq_score_mod(20.0, None, first), out, w, ws, size)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[2]) and not bool((outs[0] == 99.0).any())
    assert bool((outs[1] == 99.0).all())


def test_no_wait_ran_out():
    assert pq.pq_wait_timeouts() == 0
