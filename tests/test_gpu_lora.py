"""Adapters beside a projection against the formula in 64 bits.

Bound per element: 2^-24 |Y| + (2^-17 + 2^-32 K) |scale| sum |B| sum |A x|, the
roundings at their worst in units of u = 2^-24.  Numbers of 22 bits: 4 u each in
x and v.  Tensor core sums are truncated, 2 u a step: 8 steps a chunk of 32 in
either product, 16 u twice.  f32 sums: K / 256 chunks of a warp, 8 warps, at most
21 slices, 4 chunks of the rank; scale 1 u.  Together 74 u + K / 256 u, below
2^-17 + 2^-32 K.  The roundings average out: 1e-6 of the added term in the
2-norm."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import oracle
from gpu_util import dev, torch

pytestmark = pytest.mark.gpu
TYPES = {"f16": gq.GQ_TYPE_F16, "bf16": gq.GQ_TYPE_BF16}


class Case:
    def __init__(self, M, K, rows, rank, n_adapters, adapter, sequence, typ, q8, seed=0, pad=0):
        t = torch()
        g = np.random.default_rng(seed)
        self.__dict__.update(M=M, K=K, rows=rows, rank=rank, n_adapters=n_adapters, typ=typ, q8=q8, pad=pad)
        half = t.float16 if typ == "f16" else t.bfloat16
        self.A = t.from_numpy((g.standard_normal((n_adapters, rank, K)) * K ** -0.5).astype(np.float32)).to(half).cuda()
        self.B = t.from_numpy((g.standard_normal((n_adapters, rows, rank)) * 0.3).astype(np.float32)).to(half).cuda()
        self.scale = g.uniform(0.5, 2.0, n_adapters).astype(np.float32)
        self.adapter = np.asarray(adapter, np.int32)
        self.sequence = None if sequence is None else np.asarray(sequence, np.int32)
        self.x = g.standard_normal((M, K)).astype(np.float32)
        self.y0 = g.standard_normal((M, rows)).astype(np.float32)
        if q8:
            self.q, self.d = oracle.quantize_q8_0(self.x, M, K)
            self.x = self.q.astype(np.float64) * np.repeat(self.d.astype(np.float64), 32, -1).reshape(M, K)

    def of(self):
        """Every token's adapter, -1 for none."""
        b = np.arange(self.M) if self.sequence is None else self.sequence
        a = np.where((b >= 0) & (b < len(self.adapter)), self.adapter[np.clip(b, 0, len(self.adapter) - 1)], -1)
        return np.where((a >= 0) & (a < self.n_adapters), a, -1)

    def reference(self):
        a, b = self.A.double().cpu().numpy(), self.B.double().cpu().numpy()
        y, bound, add = self.y0.astype(np.float64), np.zeros((self.M, self.rows)), np.zeros((self.M, self.rows))
        x = self.x.astype(np.float64)
        for i, ad in enumerate(self.of()):
            if ad >= 0:
                add[i] = self.scale[ad] * (b[ad] @ (a[ad] @ x[i]))
                bound[i] = (2.0 ** -17 + 2.0 ** -32 * self.K) * self.scale[ad] * (np.abs(b[ad]) @ (np.abs(a[ad]) @ np.abs(x[i])))
        y = y + add
        return y, bound + 2.0 ** -24 * np.abs(y), add

    def run(self, in_place=False, ws=None, stream=None):
        t = torch()
        if ws is None:
            ws = t.full((gq.gq_lora_workspace_bytes(self.rank, self.K, self.M),), 0xC5, dtype=t.uint8, device="cuda")
        y0 = t.full((self.M + 1, self.rows + self.pad), -7.5, device="cuda")
        y0[:self.M, :self.rows] = dev(self.y0)
        y = y0 if in_place else t.full((self.M + 1, self.rows + 2 * self.pad), 9.5, device="cuda")
        sizes = (ws, ws.numel(), self.n_adapters, self.rank, self.rows, self.K, len(self.adapter), self.M)
        head = (self.A, self.B, TYPES[self.typ], dev(self.scale), dev(self.adapter),
                None if self.sequence is None else dev(self.sequence))
        ys = (y0[:, :self.rows], y0.stride(0), y[:, :self.rows], y.stride(0))
        if self.q8:
            gq.gq_lora_add_q8act(*head, dev(self.q), dev(self.d), *ys, *sizes, stream=stream)
        else:
            x = t.full((self.M, self.K + self.pad), float("nan"), device="cuda")
            x[:, :self.K] = dev(self.x)
            gq.gq_lora_add(*head, x[:, :self.K], x.stride(0), *ys, *sizes, stream=stream)
        t.cuda.synchronize()
        edge = -7.5 if in_place else 9.5
        assert bool((y[self.M] == edge).all()) and bool((y[:, self.rows:] == edge).all()), "written outside"
        return y[:self.M, :self.rows].cpu().numpy()

    def check(self, **kw):
        got = self.run(**kw)
        y, bound, add = self.reference()
        err = np.abs(got - y)
        assert np.all(err <= bound), (err / np.maximum(bound, 1e-300)).max()
        norm = np.linalg.norm(add)
        # the rounding of Y itself is not the product's
        assert np.linalg.norm(np.maximum(err - 2.0 ** -24 * np.abs(y), 0)) <= 1e-6 * norm
        bare = self.of() < 0
        assert np.array_equal(got[bare].view(np.int32), self.y0[bare].view(np.int32)), "rows without an adapter as they were"
        return got


def runs(lengths):
    return np.repeat(np.arange(len(lengths)), lengths)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("M,K,rows,rank", [(1, 32, 4, 8), (1, 4096, 5376, 16), (3, 288, 36, 24), (9, 5376, 260, 64), (64, 1024, 1000, 32),
                                           (70, 544, 68, 128), (33, 96, 32, 104)])
def test_decode_batches(M, K, rows, rank, typ, q8):
    g = np.random.default_rng(M)
    c = Case(M, K, rows, rank, 5, g.integers(-1, 5, M), None, typ, q8, seed=M, pad=4)
    c.check()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("lengths,K,rows,rank", [([300], 1024, 512, 16), ([17, 1, 0, 40, 260, 31], 352, 100, 40),
                                                 ([64, 64, 64], 5376, 64, 8), ([100, 29], 64, 2052, 128)])
def test_prompts(lengths, K, rows, rank, typ, q8):
    n = len(lengths)
    adapter = [(2, -1, 0, 1, 2, 0)[b % 6] for b in range(n)]
    Case(sum(lengths), K, rows, rank, 3, adapter, runs(lengths), typ, q8, seed=n, pad=8).check()


def test_every_token_its_own_adapter_and_one_for_all():
    for adapter in (np.arange(40) % 40, np.zeros(40, int), -np.ones(40, int)):
        Case(40, 256, 96, 16, 40, adapter, None, "bf16", False).check()


def test_in_place_leaves_rows_without_an_adapter_untouched():
    Case(37, 512, 128, 16, 2, [0, -1, 1], runs([10, 17, 10]), "bf16", False, pad=4).check(in_place=True)
    Case(6, 512, 128, 16, 2, [0, -1, 1, -1, -1, 0], None, "f16", True).check(in_place=True)


def test_padded_rows_and_bad_numbers():
    gq.gq_device_status()
    c = Case(20, 64, 32, 8, 2, [0, 1], [0] * 9 + [1] * 5 + [-1] * 6, "bf16", False)
    c.check()
    assert gq.gq_device_status() == gq.GQ_OK
    for adapter, sequence in (([0, 2, 1], [0] * 7 + [1] * 7 + [2] * 6), ([0, 1, 1], [0] * 7 + [3] * 7 + [2] * 6)):
        Case(20, 64, 32, 8, 2, adapter, sequence, "bf16", False).check()
        assert gq.gq_device_status() == gq.GQ_ERR_SHAPE


@pytest.mark.parametrize("what", ["x", "A", "B"])
@pytest.mark.parametrize("M,sequence", [(16, None), (320, True)])
def test_what_is_not_finite_stays_with_its_request(what, M, sequence):
    t = torch()
    seq = runs([M // 4] * 4) if sequence else None
    adapter = np.array([0, 1, 2, 1]) if sequence else np.arange(16) % 3
    c = Case(M, 128, 64, 16, 3, adapter, seq, "bf16", False)
    of = c.of()
    good, _, _ = c.reference()
    if what == "x":
        c.x[5, 3] = np.nan
        bad = np.arange(M) == 5
    elif what == "A":
        c.A[1, 2, 3] = float("inf")
        bad = of == 1
    else:
        c.B[1, 7, 2] = float("nan")
        bad = of == 1
    got = c.run()
    assert np.all(np.isfinite(got[~bad])) and np.allclose(got[~bad], good[~bad], atol=1e-4)
    assert not np.any(np.isfinite(got[bad][:, 7]))
    if what == "B":
        assert np.all(np.isfinite(np.delete(got[bad], 7, 1)))


def test_large_and_tiny_activations():
    """Two pieces of 11 bits reach down with the numbers themselves."""
    for f in (1e30, 1e-30):
        c = Case(4, 256, 32, 16, 2, [0, 1, 1, 0], None, "bf16", False)
        c.x = (c.x * np.float32(f)).astype(np.float32)
        c.y0 = (c.y0 * np.float32(f)).astype(np.float32)
        c.check()


def test_same_bits_again_and_in_a_graph():
    t = torch()
    c = Case(50, 2048, 640, 32, 7, np.arange(50) % 8 - 1, None, "f16", False)
    first = c.run()
    assert np.array_equal(first, c.run())
    ws = t.empty(gq.gq_lora_workspace_bytes(32, 2048, 50), dtype=t.uint8, device="cuda")
    x, y0, y, adapter, scale = dev(c.x), dev(c.y0), t.empty(50, 640, device="cuda"), dev(c.adapter), dev(c.scale)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        gq.gq_lora_add(c.A, c.B, TYPES["f16"], scale, adapter, None, x, 2048, y0, 640, y, 640, ws, ws.numel(), 7, 32, 640, 2048, 50, 50)
    graph.replay()
    assert np.array_equal(y.cpu().numpy(), first)
    c.adapter = np.roll(c.adapter, 5)
    adapter.copy_(dev(c.adapter))
    graph.replay()
    assert np.array_equal(y.cpu().numpy(), c.run())


def test_two_calls_at_once_with_a_workspace_each():
    t = torch()
    cs = [Case(30, 1024, 512, 16, 4, np.arange(30) % 4, None, "bf16", q8, seed=s) for s, q8 in ((1, False), (2, True))]
    alone = [c.run() for c in cs]
    streams = [t.cuda.Stream() for _ in cs]
    outs = [[], []]
    for _ in range(5):
        for i, c in enumerate(cs):
            with t.cuda.stream(streams[i]):
                outs[i].append(c.run(stream=streams[i]))
    for i in range(2):
        assert all(np.array_equal(o, alone[i]) for o in outs[i])


def test_weights_beyond_32_bits_of_elements():
    t = torch()
    n, rank, K, rows = 70, 128, 8192, 1 << 18
    A = t.zeros(n, rank, K, dtype=t.bfloat16, device="cuda")
    B = t.zeros(n, rows, rank, dtype=t.bfloat16, device="cuda")
    assert B.numel() > 1 << 31
    A[n - 1, 127, K - 1] = 2.0
    B[n - 1, rows - 1, 127] = 3.0
    x, y = t.ones(1, K, device="cuda"), t.zeros(1, rows, device="cuda")
    ws = t.empty(gq.gq_lora_workspace_bytes(rank, K, 1), dtype=t.uint8, device="cuda")
    gq.gq_lora_add(A, B, gq.GQ_TYPE_BF16, t.ones(n, device="cuda"), t.tensor([n - 1], dtype=t.int32, device="cuda"), None, x, K,
                   y, rows, y, rows, ws, ws.numel(), n, rank, rows, K, 1, 1)
    assert float(y[0, rows - 1]) == 6.0 and float(y.abs().sum()) == 6.0


@pytest.mark.parametrize("q8", [False, True])
def test_prompts_whose_tokens_lie_anywhere(q8):
    """Runs of one token, of a multiple of 16 or 32 and one more or less, over more than one round of 4096 tokens."""
    g = np.random.default_rng(5)
    sequence = g.integers(-1, 6, 700)  # nearly every token begins a run
    Case(700, 64, 36, 8, 4, [0, 3, -1, 1, 1, 2], sequence, "bf16", q8, pad=4).check()
    lengths = [1, 31, 32, 33, 1, 16, 15, 17, 64, 0, 65, 127, 3000, 1, 1024, 4096, 2]
    adapter = g.integers(-1, 3, len(lengths))
    Case(sum(lengths), 32, 20, 16, 3, adapter, runs(lengths), "f16", q8).check()
    Case(sum(lengths), 32, 20, 16, 3, adapter, runs(lengths), "f16", q8).check(in_place=True)


def test_prompts_in_a_graph_with_other_lists():
    t = torch()
    M, K, rows, rank, n_seq = 600, 256, 96, 40, 8
    c = Case(M, K, rows, rank, 3, [0, 1, -1, 2, 2, 0, 1, -1], runs([75] * 8), "bf16", False)
    ws = t.empty(gq.gq_lora_workspace_bytes(rank, K, M), dtype=t.uint8, device="cuda")
    x, y0, y, adapter, scale, sequence = dev(c.x), dev(c.y0), t.empty(M, rows, device="cuda"), dev(c.adapter), dev(c.scale), dev(c.sequence)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        for _ in range(2):
            gq.gq_lora_add(c.A, c.B, TYPES["bf16"], scale, adapter, sequence, x, K, y0, rows, y, rows, ws, ws.numel(), 3, rank, rows, K,
                           n_seq, M)
    for lengths in ([75] * 8, [1, 2, 3, 4, 90, 0, 200, 300], [593, 1, 1, 1, 1, 1, 1, 1]):
        c.sequence = runs(lengths).astype(c.sequence.dtype)
        sequence.copy_(dev(c.sequence))
        y.fill_(float("nan"))
        graph.replay()
        assert np.array_equal(y.cpu().numpy(), c.run())
        c.check()


@pytest.mark.parametrize("M,n_seq", [(7, 1), (8, 1), (9, 1), (15, 2), (16, 2), (255, 31), (255, 32), (255, 60), (256, 64), (256, 65), (260, 65)])
@pytest.mark.parametrize("q8", [False, True])
def test_both_sides_of_the_rule_for_prompts(M, n_seq, q8):
    """Few tokens a request, with a workspace of exactly the bytes asked for."""
    g = np.random.default_rng(M + n_seq)
    sequence = np.sort(g.integers(0, n_seq, M))
    Case(M, 96, 40, 24, 5, g.integers(-1, 5, n_seq), sequence, "bf16", q8, seed=n_seq).check()
