"""An attention block on libgq, prompt and decode, with its keys and values in
a paged Q8_0 cache.

One block: RMS norm -> fused q, k, v projection (Q4_0 weights) -> new keys and
values into the cache -> attention over everything cached -> output projection
-> residual.  The prompt goes through in chunks of a few tokens (the norm gives
Q8_0 activations for the contraction), later tokens one by one (matrix-vector
products); both read and write the same cache.

    python examples/attention_step.py
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import block_quantized_matvec_gq_gb300 as gq
import synth


class AttentionBlock:
    """Weights and buffers of one block; every call runs on torch's current stream.  What the library reads and writes is
    allocated once; a step makes only its result, and for a single token the normalised row (torch: the library's norm gives
    Q8_0 codes, the matrix-vector product takes f32)."""

    def __init__(self, hidden, heads, kv_heads, dim, max_tokens, n_pages, page_tokens=64, seed=7):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.page_tokens, self.n_pages = page_tokens, n_pages
        self.width = (heads + 2 * kv_heads) * dim
        self.w_qkv = self._weights(self.width, hidden, seed)
        self.w_out = self._weights(hidden, heads * dim, seed + 1)
        self.norm = torch.zeros(hidden, device="cuda")
        self.cache = torch.zeros(gq.gq_kv_cache_bytes(n_pages, page_tokens, kv_heads, dim), dtype=torch.uint8, device="cuda")
        self.attn_ws = torch.zeros(gq.gq_kv_attention_workspace_bytes(heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
        n = max(gq.gq_q4_0_gemm_workspace_bytes(k, max_tokens) for k in (hidden, heads * dim))
        self.gemm_ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        wide = max(hidden, heads * dim)
        self.codes = torch.empty(max_tokens * wide, dtype=torch.int8, device="cuda")
        self.scales = torch.empty(max_tokens * wide // 32, device="cuda")
        self.qkv = torch.empty(max_tokens, self.width, device="cuda")
        self.attn = torch.empty(max_tokens, heads * dim, device="cuda")
        self.out = torch.empty(max_tokens, hidden, device="cuda")

    @staticmethod
    def _weights(rows, cols, seed):
        w = synth.q4_0_weights(rows, cols, synth.stream(seed, 0), d_exp2=-10)
        return gq.pack(gq.GQ_FORMAT_Q4_0, torch.from_numpy(w.reshape(-1)).cuda(), rows, cols)

    def _project(self, w, x, y, rows, cols, m):
        """y = w x for m tokens of x (f32, already normalised where that is wanted)."""
        if m == 1:
            gq.gq_q4_0_matvec(w, x, y, rows, cols)
            return
        gq.gq_quantize_q8_0(x, self.codes, self.scales, cols, m)
        gq.gq_q4_0_gemm_q8act(w, self.codes, self.scales, y, self.gemm_ws, self.gemm_ws.numel(), rows, cols, m)

    def step(self, x, table, kv_len, q_start):
        """x: f32[tokens][hidden], the new tokens of all sequences; the lists say whose they are (kv_len counts them)."""
        m, h, d = x.shape[0], self.heads, self.dim
        qkv, attn = self.qkv[:m], self.attn[:m]
        if m == 1:
            r = torch.rsqrt(x.square().mean() + 1e-6)
            gq.gq_q4_0_matvec(self.w_qkv, (x * r * (self.norm + 1.0)).reshape(-1), qkv, self.width, self.hidden)
        else:
            gq.gq_rmsnorm_quantize_q8_0(x, self.norm, 1.0, 1e-6, self.codes, self.scales, self.hidden, m)
            gq.gq_q4_0_gemm_q8act(self.w_qkv, self.codes, self.scales, qkv, self.gemm_ws, self.gemm_ws.numel(), self.width,
                                  self.hidden, m)
        q, k, v = qkv[:, :h * d], qkv[:, h * d:(h + self.kv_heads) * d], qkv[:, (h + self.kv_heads) * d:]
        sizes = (self.n_pages, table.shape[1], self.page_tokens, self.kv_heads, d, table.shape[0], m)
        gq.gq_kv_append_q8_0(k, k.stride(0), v, v.stride(0), gq.GQ_TYPE_F32, self.cache, table, kv_len, q_start, *sizes)
        gq.gq_kv_attention_q8_0(q, q.stride(0), self.cache, table, kv_len, q_start, attn, attn.stride(0), gq.GQ_TYPE_F32,
                                d ** -0.5, 0.0, 0, self.attn_ws, self.attn_ws.numel(), h, *sizes)
        self._project(self.w_out, attn, self.out[:m], self.hidden, h * d, m)
        return x + self.out[:m]

    def cached(self, table, kv_len, n):
        """The first sequence's cached keys and values, read back in f32."""
        k, v = (torch.empty(n, self.kv_heads * self.dim, device="cuda") for _ in range(2))
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        gq.gq_kv_read_q8_0(self.cache, table, kv_len, start, k, k.stride(0), v, v.stride(0), gq.GQ_TYPE_F32, self.n_pages,
                           table.shape[1], self.page_tokens, self.kv_heads, self.dim, 1, n)
        return k, v


def main(prompt=75, tokens=6, hidden=1024, heads=8, kv_heads=2, dim=128):
    """A prompt in two chunks, then single tokens; returns the outputs, and checks the attention of the last step
    against the cache as it reads back."""
    g = torch.Generator(device="cuda").manual_seed(1)
    total = prompt + tokens
    block = AttentionBlock(hidden, heads, kv_heads, dim, max_tokens=prompt, n_pages=8)
    x = torch.randn(total, hidden, generator=g, device="cuda")
    table = torch.tensor([[5, 2, 7, 0]], dtype=torch.int32, device="cuda")
    outs, done = [], 0
    for n in [prompt // 2, prompt - prompt // 2] + [1] * tokens:
        kv_len = torch.tensor([done + n], dtype=torch.int32, device="cuda")
        q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        outs.append(block.step(x[done:done + n], table, kv_len, q_start))
        done += n
    k, v = block.cached(table, kv_len, total)
    q = block.qkv[0, :heads * dim].reshape(kv_heads, heads // kv_heads, dim)
    s = torch.einsum("hgd,nhd->hgn", q, k.reshape(total, kv_heads, dim)) * dim ** -0.5
    ref = torch.einsum("hgn,nhd->hgd", s.softmax(-1), v.reshape(total, kv_heads, dim)).reshape(-1)
    err = float((block.attn[0] - ref).norm() / ref.norm())
    assert err < 1e-5, err
    assert gq.gq_device_status() == gq.GQ_OK
    return torch.cat(outs), err


if __name__ == "__main__":
    y, err = main()
    print(f"{y.shape[0]} tokens through the block; attention against the cache read back: {err:.1e}")
