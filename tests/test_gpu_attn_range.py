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


def held(c, pos):
    """sum p_t s_t / sum p_t of the row at this position, which sees every token up to its own."""
    t = np.arange(pos + 1)
    pg = c.table[0, t // c.page]
    x = c.k[pg, 0, t % c.page, 0].astype(np.float64) * c.ks[pg, 0] * float(np.float32(LN2))
    p = np.exp(x - x.max())
    return float((p * 127 * np.abs(c.vs[pg, 0].astype(np.float64))).sum() / p.sum())


def check_held(c, rows, dt, ws, n_q=1, largest=1.0):
    """V scales are given over `largest`, so that f16 outputs stay in range."""
    n = int(c.len[0])
    c.vs *= np.float32(largest)
    got, ref, _ = run(c, [rows], dt, n_q, ws, scale=LN2, q=unit_q(rows, n_q, c.d))
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dt]
    bound = np.array([held(c, n - rows + r) for r in range(rows)])[:, None, None]
    tol = (4e-5 + (2.0 ** -11 if dt != "f32" else 0.0)) * bound + u * np.abs(ref) + (2.0 ** -25 if dt == "f16" else 0.0)
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the bound"


SHAPES = [(64, 1), (64, 40), (128, 1), (128, 40), (128, 12), (80, 3)]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("d,rows", SHAPES)
@pytest.mark.parametrize("more", [12, 20, 24, 40, 60, 100])
@pytest.mark.parametrize("pages", [[0], [5], [16], [2, 9, 17]])
def test_pages_of_large_scale_and_no_weight(dt, d, rows, more, pages, ws):
    # V scales 2^more above the others on pages whose tokens weigh 2^-(more + 30) of the others
    c = cache(300, 16, d, seed=more)
    c.vs[:] = 2.0 ** -more
    for j in pages:
        pg = c.table[0, j]
        c.vs[pg] = 1.0
        c.k[pg, 0, :, 0] = -127
        c.ks[pg, 0] = (more + 30) / 127.0
    check_held(c, rows, dt, ws, largest=2.0 ** (more if dt != "f16" else min(more, 8)) * 0.03)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,rows", SHAPES)
@pytest.mark.parametrize("drop", [10, 30, 60, 90])
def test_scales_fall_while_scores_rise(dt, d, rows, drop, ws):
    # from page to page the V scale falls by 2^(drop/18) and the score rises by twice that: the last pages hold the
    # weight and the smallest values
    c = cache(300, 16, d, seed=drop)
    for j in range(19):
        pg = c.table[0, j]
        c.vs[pg] = 2.0 ** (-drop * j / 18)
        c.k[pg, 0, :, 0] = 6 * j
        c.ks[pg, 0] = drop / 54.0
    check_held(c, rows, dt, ws, largest=0.03)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,rows", SHAPES)
@pytest.mark.parametrize("rise", [10, 30, 60, 100])
def test_scales_rise_while_scores_fall(dt, d, rows, rise, ws):
    # the other way round, weights falling by two thirds of the scales' rise: the last pages hold the values
    c = cache(300, 16, d, seed=rise)
    for j in range(19):
        pg = c.table[0, j]
        c.vs[pg] = 2.0 ** (rise * j / 18 - rise)
        c.k[pg, 0, :, 0] = -6 * j
        c.ks[pg, 0] = rise / 162.0
    check_held(c, rows, dt, ws, largest=0.03)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d,rows", SHAPES)
@pytest.mark.parametrize("exp", [-125, -120, -100, 100, 110])
def test_scales_at_the_ends_of_f32(dt, d, rows, exp, ws):
    c = cache(300, 16, d, seed=200 + exp)
    rng = np.random.default_rng(1)
    c.vs[:] = 2.0 ** exp * rng.uniform(1.0, 1.9, c.vs.shape)
    for t in range(300):
        put(c, t, int(rng.integers(-60, 61)), 0.05)
    check_held(c, rows, dt, ws)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows", [1, 40])
def test_nothing_but_zero_scales_then_values(dt, rows, ws):
    # pages whose V scale is 0 hold all the weight, or a part of it
    for some in (0, 9):
        c = cache(300, 16, 64, seed=5)
        c.vs[:] = 0.0
        for j in range(some, some + 4):
            pg = c.table[0, j]
            c.vs[pg] = 0.03
            c.k[pg, 0, :, 0] = -100
            c.ks[pg, 0] = 0.1
        check_held(c, rows, dt, ws)


def test_no_wait_ran_out():
    assert pq.pq_wait_timeouts() == 0
