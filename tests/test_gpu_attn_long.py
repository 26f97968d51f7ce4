"""f32 attention over long contexts, where thousands of partial sums meet.

Against 64 bits, over the norm of the output: a score of less than 6 (in powers of two) is off by
2^-22 of itself, a weight by 2^-22, and adding up to 1100 tiles' sums to one another by
sqrt(1100) * 2^-25 where each addition is rounded to nearest: together below 2e-6, however many rows
share the tiles and however long a CTA's range is.
"""
import pytest

import kvref
import quantized_weight_mat_gb300 as pq
from test_gpu_attn import dense64, setup, ws  # noqa: F401
from test_gpu_kv_cache import upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n,heads", [
    (1, 131072, (32, 8, 128)), (4, 131072, (32, 8, 128)), (64, 131072, (8, 2, 128)), (130, 60000, (32, 8, 128)),
    (64, 131072, (14, 2, 64)), (200, 30000, (16, 1, 64)), (700, 9000, (8, 2, 128)),
])
def test_sums_keep_their_bits(rows, n, heads, ws):  # noqa: F811
    import torch
    n_q, n_kv, d = heads
    c = kvref.Cache(1, [n], n_kv, 64, d, seed=rows)
    t, h = upload(c)
    q = torch.randn(rows, n_q * d, device="cuda", generator=torch.Generator("cuda").manual_seed(rows))
    out = torch.empty_like(q)
    rs = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    pq.pq_attn(h, rs, rows, "f32", q, n_q * d, n_q, d ** -0.5, 0, 0, out, n_q * d, ws, ws.numel())
    ref, _ = dense64(t, c, q.view(rows, n_q, d), n_q, torch.arange(n - rows, n, device="cuda"))
    assert float((out.double().view_as(ref) - ref).norm() / ref.norm()) <= 2e-6
