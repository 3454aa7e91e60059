"""A serving loop on libgq: requests that start, run and end share one paged cache.

Every step is made on the GPU from the requests' lengths: the lists and pages
(gq_kv_plan) -> rows of the tied embedding (gq_embed) -> one attention block,
whose q, k, v projection has an adapter per request beside it
(gq_lora_add_q8act) -> logits of each request's last token -> the next tokens
with settings of each request's own (gq_sample).

    python examples/serving_loop.py
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch

import block_quantized_matvec_gq_gb300 as gq
import synth
from attention_step import AttentionBlock

I32 = dict(dtype=torch.int32, device="cuda")


class AdaptedBlock(AttentionBlock):
    """An attention block with low-rank adapters of the q, k, v projection."""

    def __init__(self, *size, n_adapters=2, rank=16, seed=7, **kw):
        super().__init__(*size, seed=seed, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n_adapters, self.rank = n_adapters, rank
        self.lora_a = (torch.randn(n_adapters, rank, self.hidden, generator=g, device="cuda") * self.hidden ** -0.5).bfloat16()
        self.lora_b = (torch.randn(n_adapters, self.width, rank, generator=g, device="cuda") * 0.1).bfloat16()
        self.lora_scale = torch.full((n_adapters,), 0.5, device="cuda")
        self.lora_ws = torch.empty(gq.gq_lora_workspace_bytes(rank, self.hidden, self.qkv.shape[0]), dtype=torch.uint8, device="cuda")

    def step(self, x, table, kv_len, q_start, adapter, sequence):
        """x: f32[rows][hidden]; rows behind the last request (sequence -1) are computed and lead nowhere."""
        m, h, d, n = x.shape[0], self.heads, self.dim, table.shape[0]
        qkv, attn, out = self.qkv[:m], self.attn[:m], self.out[:m]
        gq.gq_rmsnorm_quantize_q8_0(x, self.norm, 1.0, 1e-6, self.codes, self.scales, self.hidden, m)
        gq.gq_q4_0_gemm_q8act(self.w_qkv, self.codes, self.scales, qkv, self.gemm_ws, self.gemm_ws.numel(), self.width,
                              self.hidden, m)
        gq.gq_lora_add_q8act(self.lora_a, self.lora_b, gq.GQ_TYPE_BF16, self.lora_scale, adapter, sequence, self.codes, self.scales,
                             qkv, qkv.stride(0), qkv, qkv.stride(0), self.lora_ws, self.lora_ws.numel(), self.n_adapters,
                             self.rank, self.width, self.hidden, n, m)
        q, k, v = qkv[:, :h * d], qkv[:, h * d:(h + self.kv_heads) * d], qkv[:, (h + self.kv_heads) * d:]
        sizes = (self.n_pages, table.shape[1], self.page_tokens, self.kv_heads, d, n, m)
        attn.zero_()  # the rows that no request owns are left as they are by the attention
        gq.gq_kv_append_q8_0(k, k.stride(0), v, v.stride(0), gq.GQ_TYPE_F32, self.cache, table, kv_len, q_start, *sizes)
        gq.gq_kv_attention_q8_0(q, q.stride(0), self.cache, table, kv_len, q_start, attn, attn.stride(0), gq.GQ_TYPE_F32,
                                d ** -0.5, 0.0, 0, self.attn_ws, self.attn_ws.numel(), h, *sizes)
        gq.gq_quantize_q8_0(attn, self.codes, self.scales, h * d, m)
        gq.gq_q4_0_gemm_q8act(self.w_out, self.codes, self.scales, out, self.gemm_ws, self.gemm_ws.numel(), self.hidden, h * d, m)
        return x + out


class Server:
    def __init__(self, slots=3, vocab=1999, hidden=512, heads=8, kv_heads=2, dim=64, rows=48, n_pages=24, max_pages=8, page=16):
        self.slots, self.vocab, self.hidden, self.rows, self.page = slots, vocab, hidden, rows, page
        self.block = AdaptedBlock(hidden, heads, kv_heads, dim, max_tokens=rows, n_pages=n_pages, page_tokens=page)
        w = synth.q8_0_weights(vocab, hidden, synth.stream(3, 0))
        self.embedding = gq.pack(gq.GQ_FORMAT_Q8_0, torch.from_numpy(w.reshape(-1)).cuda(), vocab, hidden)
        self.kv_len, self.q_start = torch.zeros(slots, **I32), torch.zeros(slots + 1, **I32)
        self.ring, self.pages = torch.tensor([0, n_pages], **I32), torch.arange(n_pages, **I32)
        self.table = torch.full((slots, max_pages), -1, **I32)
        self.slot = torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.position, self.sequence = torch.zeros(rows, **I32), torch.zeros(rows, **I32)
        self.x = torch.zeros(rows, hidden, device="cuda")
        self.logits = torch.zeros(slots, -(-vocab // 4) * 4, device="cuda")[:, :vocab]  # rows that begin on 16 bytes
        size = gq.gq_logits_topk_workspace_bytes(vocab, hidden, 1)
        self.topk_ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        self.top = torch.zeros(1, **I32), torch.zeros(1, device="cuda")
        self.sample_ws = torch.empty(gq.gq_sample_workspace_bytes(vocab, slots), dtype=torch.uint8, device="cuda")
        self.token, self.prob = torch.zeros(slots, **I32), torch.zeros(slots, device="cuda")

    def step(self, new, adapter, temperature, top_k, top_p, min_p, u):
        """new: for every slot the new tokens (a list), or None where its request has ended.  Returns every slot's next
        token, -1 where it has none."""
        n_new = torch.tensor([-1 if t is None else len(t) for t in new], **I32)
        gq.gq_kv_plan(n_new, self.kv_len, self.ring, self.pages, self.table, self.kv_len, self.q_start, self.ring, self.slot,
                      self.position, self.sequence, self.pages.numel(), self.table.shape[1], self.page, self.slots, self.rows)
        ids = [i for t in new if t for i in t]
        ids = torch.tensor(ids + [-1] * (self.rows - len(ids)), **I32)
        gq.gq_embed(gq.GQ_FORMAT_Q8_0, self.embedding, ids, self.hidden ** 0.5, self.x, self.hidden, gq.GQ_TYPE_F32, self.vocab,
                    self.hidden, self.rows)
        y = self.block.step(self.x, self.table, self.kv_len, self.q_start, adapter, self.sequence)
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
        self.logits.fill_(-float("inf"))
        row = 0
        for b, t in enumerate(new):
            if t:
                row += len(t)
                gq.gq_logits_topk(self.embedding, y[row - 1], 30.0, 1, *self.top, self.logits[b], self.topk_ws, self.topk_ws.numel(),
                                  self.vocab, self.hidden)
        gq.gq_sample(self.logits, self.logits.stride(0), gq.GQ_TYPE_F32, temperature, top_k, top_p, min_p, u, self.token, self.prob,
                     self.sample_ws, self.sample_ws.numel(), self.vocab, self.slots)
        return self.token.tolist()


def main(steps=8):
    """Three requests; one ends and another takes its place.  Returns each request's tokens and the server."""
    g = torch.Generator(device="cuda").manual_seed(2)
    s = Server()
    f32 = dict(device="cuda")
    settings = (torch.tensor([0.0, 0.8, 1.0], **f32), torch.tensor([0, 40, 0], **I32), torch.tensor([1.0, 0.9, 0.95], **f32),
                torch.tensor([0.0, 0.0, 0.02], **f32))
    adapter = torch.tensor([0, -1, 1], **I32)
    prompts = [list(range(5, 22)), [7], list(range(100, 123))]
    new, done = prompts, [[], [], []]
    for i in range(steps):
        u = torch.rand(3, generator=g, device="cuda")
        token = s.step(new, adapter, *settings, u)
        for b, t in enumerate(token):
            assert (t >= 0) == bool(new[b]) and t < s.vocab
            if t >= 0:
                done[b].append(t)
        new = [[t] if t >= 0 else [] for t in token]
        if i == 3:
            new[1] = None                       # ends: its pages return with this step
        if i == 4:
            new[1] = list(range(300, 333))      # another request in its place
    # every page is either held or free
    held = [p for b in range(3) for p in s.table[b, :-(-int(s.kv_len[b]) // s.page)].tolist()]
    first, count = s.ring.tolist()
    free = [int(s.pages[(first + i) % s.pages.numel()]) for i in range(count)]
    assert sorted(held + free) == list(range(s.pages.numel()))
    assert gq.gq_device_status() == gq.GQ_OK
    return done, s


if __name__ == "__main__":
    tokens, _ = main()
    for b, t in enumerate(tokens):
        print(f"request {b}: {t}")
