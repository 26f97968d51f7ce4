"""The attention half of a decode step of an 8B-shaped layer, for a few sequences.

    h = Wo . attention(rotate(Wqkv . x + b))

through the library's public entries: a prompt is appended to the paged 8-bit
cache and attended in one go, then single-token steps follow, each
pq_gemv_bias (QKV, Q4_K) -> pq_kv_append (q rotated in place) -> pq_attn ->
pq_gemv (O, Q4_K), all on one stream, the last attention checked against
64-bit arithmetic on the cache's own values.  Synthetic weights and inputs.

    python examples/attention_step.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import quantized_weight_mat_gb300 as pq  # noqa: E402
import synth  # noqa: E402

HIDDEN, N_Q, N_KV, D, PAGE = 4096, 32, 8, 128, 64
WIDTH = (N_Q + 2 * N_KV) * D


class Layer:
    """Weights, cache and workspace that a serving program keeps for one layer."""

    def __init__(self, n_seq: int, max_tokens: int, seed: int = 1):
        dev = torch.device("cuda")
        g = torch.Generator(device=dev).manual_seed(seed)
        self.n_seq = n_seq
        self.w_qkv = torch.from_numpy(synth.random_records("q4_k", WIDTH, HIDDEN, seed)).to(dev)
        self.w_o = torch.from_numpy(synth.random_records("q4_k", HIDDEN, N_Q * D, seed + 1)).to(dev)
        self.bias = torch.randn(WIDTH, generator=g, device=dev) * 0.1
        pages = -(-max_tokens // PAGE)
        n_pages = n_seq * pages
        self.k = torch.zeros(n_pages, N_KV, PAGE, D, dtype=torch.int8, device=dev)
        self.v = torch.zeros_like(self.k)
        self.ks = torch.zeros(n_pages, N_KV, device=dev)
        self.vs = torch.zeros_like(self.ks)
        self.table = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).reshape(n_seq, pages).contiguous()
        self.len = torch.zeros(n_seq, dtype=torch.int32, device=dev)
        self.cache = pq.pq_kv_cache(self.k, self.v, self.ks, self.vs, self.table, self.len, n_pages, N_KV, PAGE, D, n_seq, pages)
        half = D // 2
        angle = torch.arange(max_tokens, device=dev, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        self.ws = torch.empty(pq.pq_attn_ws_bytes(N_Q, N_KV, D), dtype=torch.uint8, device=dev)

    def attend(self, x: torch.Tensor, row_start=None, window: int = 0, sinks: int = 0):
        """x [rows, HIDDEN] f32 -> (attention output, layer output); row_start None: one row per sequence."""
        rows = x.shape[0]
        qkv = torch.empty(rows, WIDTH, device=x.device)
        pq.pq_gemv_bias("q4_k", self.w_qkv, WIDTH, HIDDEN, x, rows, self.bias, qkv)
        self.len += 1 if row_start is None else (row_start[1:] - row_start[:-1])
        k, v = qkv[:, N_Q * D:], qkv[:, (N_Q + N_KV) * D:]
        pq.pq_kv_append(self.cache, row_start, rows, "f32", k, WIDTH, v, WIDTH, qkv, WIDTH, N_Q, qkv, WIDTH,
                        self.cos, self.sin, self.cos.shape[0], D, "half")
        att = torch.empty(rows, N_Q * D, device=x.device)
        pq.pq_attn(self.cache, row_start, rows, "f32", qkv, WIDTH, N_Q, D ** -0.5, window, sinks, att, N_Q * D,
                   self.ws, self.ws.numel())
        out = torch.empty(rows, HIDDEN, device=x.device)
        pq.pq_gemv("q4_k", self.w_o, HIDDEN, N_Q * D, att, rows, out)
        return qkv, att, out


def check(layer: Layer, qkv: torch.Tensor, att: torch.Tensor) -> float:
    """Largest error of the last single-token attention against 64 bits, over the largest |v|."""
    worst = 0.0
    for s, n in enumerate(layer.len.tolist()):
        start = torch.zeros(layer.n_seq + 1, dtype=torch.int32, device=att.device)
        start[s + 1:] = n
        k = torch.empty(n, N_KV * D, device=att.device)
        v = torch.empty_like(k)
        pq.pq_kv_gather(layer.cache, start, n, "f32", k, N_KV * D, v, N_KV * D)
        q = qkv[s, :N_Q * D].double().view(N_KV, N_Q // N_KV, D)
        kd, vd = (t.double().view(n, N_KV, D).transpose(0, 1) for t in (k, v))
        ref = torch.softmax(q @ kd.transpose(1, 2) * D ** -0.5, -1) @ vd
        worst = max(worst, float((att[s].double().view_as(ref) - ref).abs().max() / vd.abs().max()))
    return worst


def main(prompt=(37, 150, 4), steps: int = 5) -> float:
    layer = Layer(len(prompt), max(prompt) + steps)
    rows = sum(prompt)
    start = torch.tensor([sum(prompt[:i]) for i in range(len(prompt) + 1)], dtype=torch.int32, device="cuda")
    x = torch.randn(rows, HIDDEN, device="cuda")
    layer.attend(x, start)
    for _ in range(steps):
        qkv, att, out = layer.attend(torch.randn(len(prompt), HIDDEN, device="cuda"))
    assert torch.isfinite(out).all()
    err = check(layer, qkv, att)
    print(f"{rows} prompt rows, {steps} steps: lengths {layer.len.tolist()}, attention within {err:.2e} of max|v|")
    return err


if __name__ == "__main__":
    main()
