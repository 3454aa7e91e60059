"""Calls of the serving operators that run at the same time on two streams, each with its own workspace.

Everything is allocated before; a kernel that idles holds both streams back until all calls are in their queues, and
nothing waits for the GPU before the last call.  Every call has outputs of its own, which have to be those of the same call
alone, bit by bit."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import oracle
import synth
from gpu_util import dev, packed, torch

pytestmark = pytest.mark.gpu
CALLS = 24


def sampling(seed, flat, n=30, vocab=40000):
    t = torch()
    g = np.random.default_rng(seed)
    x = dev((g.standard_normal((n, vocab)) * 0.3 if flat else g.exponential(1.5, (n, vocab))).astype(np.float32))
    u, p = dev(g.random(n).astype(np.float32)), t.full((n,), 0.9, device="cuda")
    m = t.full((n,), 0.2 if flat else 0.0, device="cuda")
    ws = t.zeros(gq.gq_sample_workspace_bytes(vocab, n), dtype=t.uint8, device="cuda")

    def outputs():
        return t.zeros(n, dtype=t.int32, device="cuda"), t.zeros(n, device="cuda")

    def call(out):
        gq.gq_sample(x, vocab, gq.GQ_TYPE_F32, None, None, p, m, u, *out, ws, ws.numel(), vocab, n)

    return call, outputs


def adapters(seed, prompts, q8, M=96, K=2048, rows=1024, rank=32, n_adapters=6):
    t = torch()
    g = np.random.default_rng(seed)
    n_seq = 5 if prompts else M
    A = (t.from_numpy(g.standard_normal((n_adapters, rank, K)) * K ** -0.5)).bfloat16().cuda()
    B = (t.from_numpy(g.standard_normal((n_adapters, rows, rank)) * 0.3)).bfloat16().cuda()
    scale, adapter = dev(g.uniform(0.5, 2.0, n_adapters).astype(np.float32)), dev(g.integers(-1, n_adapters, n_seq).astype(np.int32))
    sequence = dev(np.sort(g.integers(0, n_seq, M)).astype(np.int32)) if prompts else None
    x = g.standard_normal((M, K)).astype(np.float32)
    y0 = dev(g.standard_normal((M, rows)).astype(np.float32))
    ws = t.zeros(gq.gq_lora_workspace_bytes(rank, K, M), dtype=t.uint8, device="cuda")
    act = tuple(map(dev, oracle.quantize_q8_0(x, M, K))) if q8 else (dev(x), K)
    entry = gq.gq_lora_add_q8act if q8 else gq.gq_lora_add

    def outputs():
        return (t.zeros(M, rows, device="cuda"),)

    def call(out):
        entry(A, B, gq.GQ_TYPE_BF16, scale, adapter, sequence, *act, y0, rows, out[0], rows, ws, ws.numel(), n_adapters, rank, rows, K,
              n_seq, M)

    return call, outputs


def lists(seed, n_seq=700, page=16, max_pages=40):
    t = torch()
    g = np.random.default_rng(seed)
    kv = g.integers(0, 400, n_seq)
    new = np.where(g.random(n_seq) < 0.1, -1, g.integers(0, 40, n_seq))
    tokens, n_pages = int(np.maximum(new, 0).sum()), n_seq * max_pages
    have = -(-kv // page)
    table = np.full((n_seq, max_pages), -1, np.int32)
    table[np.arange(max_pages) < have[:, None]] = np.arange(have.sum())
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - have.sum()] = np.arange(have.sum(), n_pages)
    n_new, kv_in, ring_in = dev(new.astype(np.int32)), dev(kv.astype(np.int32)), dev(np.array([0, n_pages - have.sum()], np.int32))

    def outputs():
        i32 = dict(dtype=t.int32, device="cuda")
        return (dev(free), dev(table), t.zeros(n_seq, **i32), t.zeros(n_seq + 1, **i32), t.zeros(2, **i32),
                t.zeros(tokens, dtype=t.int64, device="cuda"), t.zeros(tokens, **i32), t.zeros(tokens, **i32))

    def call(out):
        gq.gq_kv_plan(n_new, kv_in, ring_in, *out, n_pages, max_pages, page, n_seq, tokens)

    return call, outputs


def rows_of_a_table(seed, rows=3000, K=512, M=700):
    t = torch()
    g = np.random.default_rng(seed)
    W = packed(gq.GQ_FORMAT_Q8_0, synth.q8_0_weights(rows, K, synth.stream(seed, 0)), rows, K)
    ids = dev(g.integers(0, rows, M).astype(np.int32))

    def outputs():
        return (t.zeros(M, K, device="cuda"),)

    def call(out):
        gq.gq_embed(gq.GQ_FORMAT_Q8_0, W, ids, 2.0, out[0], K, gq.GQ_TYPE_F32, rows, K, M)

    return call, outputs


KINDS = {"settled": lambda s: sampling(s, False), "searched": lambda s: sampling(s, True),
         "decode": lambda s: adapters(s, False, False), "prompts": lambda s: adapters(s, True, True),
         "lists": lists, "rows": rows_of_a_table}


@pytest.mark.parametrize("a,b", [("settled", "settled"), ("searched", "searched"), ("settled", "searched"), ("decode", "decode"),
                                 ("prompts", "prompts"), ("decode", "prompts"), ("lists", "lists"), ("rows", "lists"),
                                 ("searched", "prompts")])
def test_two_streams_at_once(a, b):
    t = torch()
    jobs = [KINDS[a](21), KINDS[b](22)]
    alone = [outputs() for _, outputs in jobs]
    for (call, _), out in zip(jobs, alone):
        call(out)
    got = [[outputs() for _ in range(CALLS)] for _, outputs in jobs]
    streams = [t.cuda.Stream() for _ in jobs]
    t.cuda.synchronize()
    for s in streams:
        with t.cuda.stream(s):
            t.cuda._sleep(10_000_000)  # some 5 ms
    for i in range(CALLS):
        for j, s in enumerate(streams):
            with t.cuda.stream(s):
                jobs[j][0](got[j][i])
    t.cuda.synchronize()
    for want, outs in zip(alone, got):
        for out in outs:
            assert all(bool(t.equal(x, y)) for x, y in zip(out, want))
    assert gq.gq_device_status() == gq.GQ_OK
