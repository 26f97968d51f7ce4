"""Chains of small calls on the generic kernels, which may be scheduled beside
their predecessor (grids of at most one block per SM): every input, a bias and
a weight's scales among them, is what the call before wrote.

Before each run the outputs hold NaN, as in test_gpu_chains.py.
"""
from __future__ import annotations

import numpy as np
import pytest

import quantized_weight_mat_gb300 as pq
import synth

pytestmark = pytest.mark.gpu
N = 1024          # 128 blocks of 8 rows: fewer than an SM each


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


@pytest.fixture
def static_weights():
    before = pq.pq_set_weight_prefetch(True)
    yield
    pq.pq_set_weight_prefetch(bool(before))


def repeated(call, outs, runs=20):
    """`call(wait)` fills `outs`; the same bits whether or not every step is waited for."""
    import torch

    def once(wait):
        for y in outs:
            y.fill_(float("nan"))
        torch.cuda.synchronize()
        call(wait)
        torch.cuda.synchronize()
        return [y.view(torch.int32).clone() for y in outs]
    want = once(True)
    assert all(bool(torch.isfinite(y).all()) for y in outs)
    for _ in range(runs):
        assert all(torch.equal(a, b) for a, b in zip(once(False), want))


def mat(fmt, n, k, seed):
    import torch
    return torch.from_numpy(synth.random_records(fmt, n, k, seed)).cuda()


def chain_of(fmt, batch, kernel, k=N):
    import torch
    ws = [mat(fmt, N, k if j == 0 else N, j) for j in range(4)]
    x = torch.from_numpy(synth.normal_x(batch, k, 9).reshape(-1)).cuda()
    ys = [torch.empty(batch * N, device="cuda") for _ in ws]

    def call(wait):
        cur, kk = x, k
        for w, y in zip(ws, ys):
            pq.pq_gemv_kernel(fmt, w, N, kk, cur, batch, y, kernel=kernel)
            cur, kk = y, N
            if wait:
                torch.cuda.synchronize()
    repeated(call, ys)


@pytest.mark.parametrize("batch", [1, 2, 3, 4])
@pytest.mark.parametrize("fmt", ["q4_k", "q6_k", "q8_0", "q5_k", "q3_k", "q2_k", "i8_row", "i4_row"])
def test_generic_calls(fmt, batch):
    chain_of(fmt, batch, "generic")


@pytest.mark.parametrize("batch", [1, 4])
def test_short_rows_with_static_weights(batch, static_weights):
    chain_of("q8_0", batch, "auto")


@pytest.mark.parametrize("fmt,kernel", [("i8_row", "generic"), ("i8_row", "auto"), ("i4_row", "generic")])
def test_row_scales_written_by_the_call_before(fmt, kernel):
    # the first call's y is the second matrix's scales
    import torch
    a, b = mat("q4_k", N, N, 1), mat(fmt, N, N, 2)
    at = N * N if fmt == "i8_row" else N * N // 2
    x = torch.from_numpy(synth.normal_x(1, N, 3).reshape(-1)).cuda()
    scales, y = b[at:].view(torch.float32), torch.empty(N, device="cuda")

    def call(wait):
        pq.pq_gemv_kernel("q4_k", a, N, N, x, 1, scales, kernel="generic")
        if wait:
            torch.cuda.synchronize()
        pq.pq_gemv_kernel(fmt, b, N, N, x, 1, y, kernel=kernel)
    repeated(call, [scales, y])


@pytest.mark.parametrize("fmt,batch", [("q4_k", 1), ("q4_k", 8), ("q4_k", 16), ("i8_row", 1), ("q8_0", 1)])
def test_bias_written_by_the_call_before(fmt, batch):
    import torch
    n, k = 4096, 4096
    a, b = mat("q4_k", n, k, 1), mat(fmt, n, k, 2)
    x = torch.from_numpy(synth.normal_x(batch, k, 3).reshape(-1)).cuda()
    bias, y = torch.empty(n, device="cuda"), torch.empty(batch * n, device="cuda")

    def call(wait):
        pq.pq_gemv("q4_k", a, n, k, x, 1, bias)
        if wait:
            torch.cuda.synchronize()
        pq.pq_gemv_bias(fmt, b, n, k, x, batch, bias, y)
    repeated(call, [bias, y])


@pytest.mark.parametrize("fmt", ["q8_0", "i8_row", "q6_k"])
def test_attention_then_a_generic_call(fmt):
    import torch
    n_seq, n_kv, page, d, n_q = 4, 2, 16, 64, 16
    g = torch.Generator().manual_seed(5)
    codes = [torch.randint(-127, 128, (n_seq * 4, n_kv, page, d), generator=g).to(torch.int8).cuda() for _ in range(2)]
    scales = [torch.full((n_seq * 4, n_kv), 0.03, device="cuda") for _ in range(2)]
    table = torch.randperm(n_seq * 4, generator=g).to(torch.int32).reshape(n_seq, 4).contiguous().cuda()
    lens = torch.tensor([1, 17, 40, 64], dtype=torch.int32, device="cuda")
    q = torch.randn((n_seq, n_q * d), generator=g).cuda()
    ws = torch.empty(pq.pq_attn_ws_bytes(n_q, n_kv, d), dtype=torch.uint8, device="cuda")
    c = pq.pq_kv_cache(codes[0], codes[1], scales[0], scales[1], table, lens, n_seq * 4, n_kv, page, d, n_seq, 4)
    w = mat(fmt, N, n_q * d, 4)
    att, y = torch.empty(n_seq * n_q * d, device="cuda"), torch.empty(n_seq * N, device="cuda")

    def call(wait):
        pq.pq_attn(c, None, n_seq, "f32", q, n_q * d, n_q, d ** -0.5, 0, 0, att, n_q * d, ws, ws.numel())
        if wait:
            torch.cuda.synchronize()
        pq.pq_gemv_kernel(fmt, w, N, n_q * d, att, n_seq, y, kernel="generic")
    repeated(call, [att, y])
