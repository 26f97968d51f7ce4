"""Attention whose softmax is decided by one token, or a few that tie, for every row and element.

Scores spread over thousands, so that they carry an f32 error of their own: delta, below 2^-20 of the
largest sum |q k| scale (see test_gpu_attn.py).  Tokens more than 17 + 2 delta below the largest score weigh
at most e^-17 each, 400 of them less than 2e-5 of the output, which is inside the bound
    (4e-5 [+ 2^-11]) * max|v| + u * |v|;
the others average, so that every element lies between the least and the largest of theirs.
"""
import numpy as np
import pytest

import kvref
import quantized_weight_mat_gb300 as pq
from test_gpu_attn import DTS, run, setup, ws  # noqa: F401
from test_gpu_kv_cache import tdt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 2, 128), (6, 2, 48)])
@pytest.mark.parametrize("news", [None, [3, 5], [150, 3], [300, 37]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 5)])
def test_one_token_takes_all_of_every_row(dt, heads, news, window, sinks, ws):  # noqa: F811
    import torch
    n_q, n_kv, d = heads
    lens, scale = [400, 37], d ** -0.5
    c = kvref.Cache(2, lens, n_kv, 32, d, seed=9)
    got, _, _ = run(c, news, dt, n_q, ws, qmul=3000.0, window=window, sinks=sinks)
    row_start = None if news is None else np.concatenate([[0], np.cumsum(news)])
    rows, w = got.shape[0], n_q * d
    q = torch.from_numpy(np.random.default_rng(1).normal(0, 3000.0, (rows, w + 16)).astype(np.float32)).to(tdt(dt)).float().numpy()
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    one = 0
    for r, (s, pos) in enumerate(kvref.places(c, row_start, rows)):
        t = np.arange(pos + 1)
        if window:
            t = t[(pos - t < window) | (t < sinks)]
        pg = c.table[s, t // c.page]
        for h in range(n_q):
            kvh, qh = h // (n_q // n_kv), q[r, h * d:(h + 1) * d].astype(np.float64)
            k = c.k[pg, kvh, t % c.page].astype(np.float64) * c.ks[pg, kvh][:, None]
            v = c.v[pg, kvh, t % c.page].astype(np.float64) * c.vs[pg, kvh][:, None]
            x = k @ qh * scale
            delta = 2.0 ** -20 * np.abs(k * qh).sum(axis=1).max() * scale
            near = v[x >= x.max() - 17.0 - 2 * delta]
            one += len(near) == 1
            tol = (4e-5 + (2.0 ** -11 if dt != "f32" else 0.0)) * np.abs(v).max() + u * np.abs(near).max(axis=0)
            assert (got[r, h] >= near.min(axis=0) - tol).all() and (got[r, h] <= near.max(axis=0) + tol).all(), (r, h)
    assert one > 0.85 * rows * n_q


def test_no_wait_ran_out():
    assert pq.pq_wait_timeouts() == 0
