"""Back-to-back calls whose every input is the previous call's output.

Before each run the outputs hold NaN, so a kernel that is scheduled beside its
predecessor and reads before that one has written is seen in every repetition.
"""
from __future__ import annotations

import numpy as np
import pytest

import quantized_weight_mat_gb300 as pq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup(cuda_ok):
    from quantized_weight_mat_gb300 import build
    build.build()


def q4_k(n, k, seed):
    import torch
    w = np.random.default_rng(seed).integers(0, 256, (n * k // 256, 144), dtype=np.uint8)
    w[:, 0:4] = np.array([1e-3, 1e-3], np.float16).view(np.uint8)
    return torch.from_numpy(w.reshape(-1)).cuda()


@pytest.mark.parametrize("batch", [1, 2, 4, 5, 8, 12, 32])
def test_a_call_reads_finished_outputs(batch):
    import torch
    shapes = [(14336, 4096), (4096, 14336), (4096, 4096), (4096, 4096)]
    ws = [q4_k(n, k, j) for j, (n, k) in enumerate(shapes)]
    x = torch.from_numpy(np.random.default_rng(9).normal(size=batch * 4096).astype(np.float32)).cuda()
    ys = [torch.empty(batch * n, device="cuda") for n, _ in shapes]

    def chain(wait):
        cur = x
        for w, (n, k), y in zip(ws, shapes, ys):
            pq.pq_gemv("q4_k", w, n, k, cur, batch, y)
            cur = y
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [y.view(torch.int32).clone() for y in ys]

    want = chain(True)
    for _ in range(20):
        for y in ys:
            y.fill_(float("nan"))
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


def test_lengths_and_table_written_by_the_call_before():
    # a copy kernel's lengths, table and rows are read by the append and the attention right after it
    import torch
    n_seq, n_kv, page, d, n_q, blocks = 64, 2, 16, 64, 8, 8
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(n_seq * blocks, generator=g).to(torch.int32).cuda()
    lens = torch.randint(2, blocks * page, (n_seq,), generator=g).to(torch.int32).cuda()
    rows = torch.randn((n_seq, (n_q + 2 * n_kv) * d), generator=g).to(torch.bfloat16).cuda()
    ws = torch.empty(pq.pq_attn_ws_bytes(n_q, n_kv, d), dtype=torch.uint8, device="cuda")
    w = rows.shape[1]

    def run(wait):
        codes = [torch.zeros(n_seq * blocks * n_kv * page * d, dtype=torch.int8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(n_seq * blocks * n_kv, device="cuda") for _ in range(2)]
        t, n, r = torch.full_like(table, -1), torch.zeros_like(lens), torch.full_like(rows, float("nan"))
        out = torch.full((n_seq, n_q * d), float("nan"), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        t.copy_(table)
        n.copy_(lens)
        r.copy_(rows)
        c = pq.pq_kv_cache(codes[0], codes[1], scales[0], scales[1], t, n, n_seq * blocks, n_kv, page, d, n_seq, blocks)
        at = r.data_ptr()
        for call in range(2):
            if wait:
                torch.cuda.synchronize()
            if call == 0:
                pq.pq_kv_append(c, None, n_seq, "bf16", at + 2 * n_q * d, w, at + 2 * (n_q + n_kv) * d, w)
            else:
                pq.pq_attn(c, None, n_seq, "bf16", at, w, n_q, 0.125, 0, 0, out, n_q * d, ws, ws.numel())
        torch.cuda.synchronize()
        return torch.cat([x.view(torch.uint8).reshape(-1) for x in (out, codes[0], codes[1], scales[0], scales[1])])

    want = run(True)
    for _ in range(10):
        assert torch.equal(run(False), want)
