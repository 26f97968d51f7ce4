"""Attention over the paged 8-bit cache where scores or page scales span far more than fp16 does.

q is one unit vector and the softmax scale ln 2, so that a token's score is
code * page scale in powers of two and every weight of the 64-bit reference is
known by construction.  Bounds as in test_gpu_attn.py; where page scales
differ widely they are relative to what the row's weights make of them,
    |out - ref| <= (4e-5 [+ 2^-11]) * sum p_t s_t / sum p_t + u * |ref|,
s_t = 127 times the V scale of the token's page, the largest value it can hold.
"""
import numpy as np
import pytest

import kvref
import quantized_weight_mat_gb300 as pq
from test_gpu_attn import DTS, check, run

pytestmark = pytest.mark.gpu
LN2 = float(np.log(2.0))


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def ws():
    import torch
    return torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")


def cache(n, page, d, seed):
    """One sequence and kv head whose scores are set page by page; V codes are random."""
    c = kvref.Cache(1, [n], 1, page, d, seed=seed)
    c.k[:] = 0
    return c


def put(c, token, code, step):
    """Score code * step for a token; step holds for its whole page."""
    pg = c.table[0, token // c.page]
    c.k[pg, 0, token % c.page, 0] = code
    c.ks[pg, 0] = step


def unit_q(rows, n_q, d, pad=16):
    import torch
    q = torch.zeros(rows, n_q * d + pad)
    q[:, 0:n_q * d:d] = 1.0
    return q


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,end", [(40, 300), (40, 256), (1, 300)])
@pytest.mark.parametrize("top", [14.0, 17.5, 20.25, 22.5, 24.0, 24.5, 24.75, 25.0, 25.25, 27.0])
def test_the_maximum_jumps_inside_a_tile(dt, d, rows, end, top, ws):
    # tokens 128..191 weigh up to just under 2^15 together, then one token is 2^top: the earlier ones still count for
    # 2^(14.9 - top) of the sum, which is all that most elements of the output hold
    c = cache(end, 64, d, seed=3)
    for t in range(128, 192):
        put(c, t, 89, 0.1)
        c.v[c.table[0, 2], 0, t % 64] = 127
    put(c, 192, int(top * 4), 0.25)
    c.v[c.table[0, 3:], 0] = 0
    c.v[c.table[0, 3], 0, 0, :8] = 127
    c.vs[:] = 0.03
    check(*run(c, [rows], dt, 1, ws, scale=LN2, q=unit_q(rows, 1, d)), dt)


def test_no_wait_ran_out():
    assert pq.pq_wait_timeouts() == 0
