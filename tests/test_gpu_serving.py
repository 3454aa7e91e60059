"""A serving step's operators together: the example loop, and a step's pieces
against one another."""

import os
import sys

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
from gpu_util import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_loop_runs_and_gives_the_same_tokens_again():
    import serving_loop
    a, s = serving_loop.main()
    b, _ = serving_loop.main()
    assert a == b
    # request 1: a token for its prompt and three more, none while it ends, then its successor's
    assert [len(t) for t in a] == [8, 7, 8]
    assert s.kv_len.tolist() == [17 + 7, 33 + 2, 23 + 7]


def test_the_greedy_request_follows_its_logits():
    import serving_loop
    _, s = serving_loop.main(steps=3)
    assert int(s.token[0]) == int(s.logits[0].argmax()) and float(s.prob[0]) == 1.0
    p = (s.logits[2].double()).softmax(-1)
    kept = p >= 0.02 * p.max()
    order = p.sort(descending=True)
    n = int((order.values.cumsum(-1) < 0.95).sum()) + 1
    assert int(s.token[2]) in order.indices[:n].tolist() and bool(kept[int(s.token[2])])


def test_a_captured_step_is_replayed_while_requests_grow():
    """Plan, embedding, adapters and sampling in one graph of a fixed number of rows, each step's tokens fed to the next."""
    t = torch()
    n, rows, vocab, hidden, pages = 4, 8, 700, 256, 40
    i32 = dict(dtype=t.int32, device="cuda")
    g = t.Generator(device="cuda").manual_seed(1)
    W = t.randint(0, 256, (gq.gq_packed_bytes(1, vocab, hidden),), dtype=t.uint8, device="cuda", generator=g)
    W[vocab * hidden:] = (t.rand(vocab * hidden // 32, device="cuda", generator=g) * 0.01).half().view(t.uint8)
    A = (t.randn(2, 8, hidden, device="cuda", generator=g) * hidden ** -0.5).half()
    B = t.randn(2, vocab + 4 - vocab % 4, 8, device="cuda", generator=g).half()
    width = B.shape[1]
    kv, ring, table = t.zeros(n, **i32), t.tensor([0, pages], **i32), t.full((n, 6), -1, **i32)
    free, q_start, new = t.arange(pages, **i32), t.zeros(n + 1, **i32), t.ones(n, **i32)
    seq, ids, token = t.zeros(rows, **i32), t.full((rows,), -1, **i32), t.zeros(n, **i32)
    x, y0, y = t.zeros(rows, hidden, device="cuda"), t.zeros(rows, width, device="cuda"), t.zeros(rows, width, device="cuda")
    adapter, scale, u = t.tensor([0, 1, -1, 1], **i32), t.ones(2, device="cuda"), t.rand(n, device="cuda", generator=g)
    lws = t.empty(gq.gq_lora_workspace_bytes(8, hidden, rows), dtype=t.uint8, device="cuda")
    sws = t.empty(gq.gq_sample_workspace_bytes(vocab, n), dtype=t.uint8, device="cuda")
    ids[:n] = t.tensor([1, 2, 3, 4])

    def step():
        gq.gq_kv_plan(new, kv, ring, free, table, kv, q_start, ring, None, None, seq, pages, 6, 16, n, rows)
        gq.gq_embed(1, W, ids, 1.0, x, hidden, 0, vocab, hidden, rows)
        gq.gq_lora_add(A, B, gq.GQ_TYPE_F16, scale, adapter, seq, x, hidden, y0, width, y, width, lws, lws.numel(), 2, 8, width,
                       hidden, n, rows)
        gq.gq_sample(y[:n, :vocab], width, 0, None, None, None, None, u, token, None, sws, sws.numel(), vocab, n)
        ids[:n].copy_(token)

    def plain(ids_now):
        out = []
        for b in range(n):
            w = W[:vocab * hidden].view(vocab, hidden)[ids_now[b]].double() - 128
            d = W[vocab * hidden:].view(t.float16).view(vocab, hidden // 32)[ids_now[b]].double()
            row = (w.view(-1, 32) * d[:, None]).reshape(-1)
            l = t.zeros(vocab, dtype=t.float64, device="cuda")
            if int(adapter[b]) >= 0:
                a = int(adapter[b])
                l = (B[a].double() @ (A[a].double() @ row))[:vocab]
            v, order = l.sort(descending=True, stable=True)
            p = v.softmax(-1).cumsum(-1)
            j = int((p <= float(u[b])).sum())
            # the neighbours too, where u is within 1e-5 of a running probability: logits are off by 1e-6 of some 10
            out.append({int(order[min(max(k, 0), vocab - 1)]) for k in (j - 1, j, j + 1)
                        if k == j or abs(float(p[min(max(min(k, j), 0), vocab - 1)]) - float(u[b])) < 1e-5})
        return out

    step()
    t.cuda.synchronize()
    kv.zero_(), table.fill_(-1), ids[:n].copy_(t.tensor([1, 2, 3, 4]))
    ring.copy_(t.tensor([0, pages])), free.copy_(t.arange(pages))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    now = [1, 2, 3, 4]
    gq.gq_device_status()
    for i in range(40):
        graph.replay()
        got, want = token.tolist(), plain(now)
        assert all(a in w for a, w in zip(got, want)), (i, got, want)
        assert kv.tolist() == [i + 1] * n and seq.tolist() == [0, 1, 2, 3] + [-1] * 4
        now = got
    assert gq.gq_device_status() == gq.GQ_OK
