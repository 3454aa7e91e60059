"""A step's lists against a plain walk over the requests; refused steps change
nothing; pages are never lost or shared over many steps; the lists lead the
cache's kernels."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
from gpu_util import dev, torch

pytestmark = pytest.mark.gpu


class State:
    """Requests of random lengths with pages in random order, the rest of the pages in the ring."""

    def __init__(self, n, page, kv, spare, room, seed=0):
        g = np.random.default_rng(seed)
        self.g, self.n, self.page = g, n, page
        self.kv = g.integers(0, kv + 1, n).astype(np.int32)
        have = -(-self.kv // page)
        self.max_pages = -(-(kv + room) // page) + 1
        self.n_pages = int(have.sum()) + spare
        order = g.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((n, self.max_pages), -9, np.int32)
        at = 0
        for b in range(n):
            self.table[b, :have[b]] = order[at:at + have[b]]
            at += have[b]
        self.first = int(g.integers(0, self.n_pages))
        self.count = spare
        self.free = np.full(self.n_pages, -5, np.int32)
        self.free[(self.first + np.arange(spare)) % self.n_pages] = order[at:]

    def plan(self, new, n_tokens):
        """The definition, request by request."""
        table, free = self.table.copy(), self.free.copy()
        first, end = self.first, self.first + self.count
        kv, q_start, rows = [], [0], []
        for b, (n, old) in enumerate(zip(new, self.kv)):
            n, old = int(n), int(old)
            have = -(-old // self.page)
            if n < 0:
                for j in range(have):
                    free[end % self.n_pages] = table[b, j]
                    end += 1
                kv.append(0)
                q_start.append(q_start[-1])
                continue
            for j in range(have, -(-(old + n) // self.page)):
                table[b, j] = free[first % self.n_pages]
                first += 1
            rows += [(int(table[b, x // self.page]) * self.page + x % self.page, x, b) for x in range(old, old + n)]
            kv.append(old + n)
            q_start.append(q_start[-1] + n)
        rows += [(-1, -1, -1)] * (n_tokens - len(rows))
        rows = np.array(rows, np.int64).reshape(-1, 3)
        return dict(kv_len=np.array(kv), q_start=np.array(q_start), table=table, free=free,
                    ring=np.array([first % self.n_pages, end - first]), slot=rows[:, 0], position=rows[:, 1], sequence=rows[:, 2])


def run(s, new, n_tokens, in_place=False, kv=None, ring=None, table=None, free=None, tokens=True):
    t = torch()
    i32 = lambda v: dev(np.asarray(v, np.int32))  # noqa: E731
    kv, ring = i32(s.kv if kv is None else kv), i32((s.first, s.count) if ring is None else ring)
    table, free = i32(s.table if table is None else table), i32(s.free if free is None else free)
    out = dict(kv_len=kv if in_place else t.full((s.n,), 77, dtype=t.int32, device="cuda"),
               ring=ring if in_place else t.full((2,), 77, dtype=t.int32, device="cuda"),
               q_start=t.full((s.n + 1,), 77, dtype=t.int32, device="cuda"), table=table, free=free)
    tok = dict(slot=t.full((n_tokens + 1,), 77, dtype=t.int64, device="cuda"),
               position=t.full((n_tokens + 1,), 77, dtype=t.int32, device="cuda"),
               sequence=t.full((n_tokens + 1,), 77, dtype=t.int32, device="cuda"))
    gq.gq_kv_plan(i32(new), kv, ring, free, table, out["kv_len"], out["q_start"], out["ring"],
                  *(tok.values() if tokens else (None,) * 3), s.n_pages, s.max_pages, s.page, s.n, n_tokens)
    got = {k: v.cpu().numpy() for k, v in out.items()}
    if tokens:
        for k, v in tok.items():
            assert int(v[n_tokens]) == 77, "written outside"
            got[k] = v[:n_tokens].cpu().numpy()
    return got


def same(got, want):
    for k, v in got.items():
        assert np.array_equal(v, want[k]), k


def step(g, n, most, ended=0.1):
    new = g.integers(0, most + 1, n)
    new[g.random(n) < ended] = -1
    return new


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,page,kv,most", [(1, 16, 0, 1), (1, 4096, 5000, 3000), (3, 16, 33, 1), (64, 64, 900, 1), (100, 48, 100, 200),
                                            (1000, 16, 50, 60), (1025, 32, 64, 3), (8192, 16, 20, 2)])
def test_lists(n, page, kv, most, in_place):
    s = State(n, page, kv, spare=n * (most // page + 1) + 3, room=most, seed=n)
    new = step(s.g, n, most)
    total = int(np.maximum(new, 0).sum())
    gq.gq_device_status()
    for n_tokens in (total, total + 37):
        same(run(s, new, n_tokens, in_place), s.plan(new, n_tokens))
    same(run(s, new, total, in_place, tokens=False), s.plan(new, total))
    assert gq.gq_device_status() == gq.GQ_OK


def test_all_end_and_nothing_new():
    s = State(50, 16, 200, spare=4, room=0)
    same(run(s, np.full(50, -1), 0), s.plan(np.full(50, -1), 0))
    same(run(s, np.zeros(50), 3), s.plan(np.zeros(50), 3))
    # a step that takes the very last free page
    s = State(1, 16, 0, spare=2, room=32)
    same(run(s, [32], 32), s.plan([32], 32))


def test_refused_steps_change_nothing():
    s = State(6, 16, 40, spare=3, room=64, seed=3)
    s.kv[2], s.kv[4] = 16, 32
    good = np.array([1, 0, 1, -1, 0, 1])
    big = np.array([64, 64, 64, 64, 64, 64])

    def refused(new, n_tokens, **kw):
        gq.gq_device_status()
        got = run(s, new, n_tokens, **kw)
        assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
        assert np.array_equal(got["kv_len"], kw.get("kv", s.kv)) and np.all(got["q_start"] == 0)
        assert np.array_equal(got["ring"], kw.get("ring", (s.first, s.count)))
        assert np.array_equal(got["table"], s.table) and np.array_equal(got["free"], s.free)
        assert all(np.all(got[x] == -1) for x in ("slot", "position", "sequence"))

    for in_place in (False, True):
        refused(good, 2, in_place=in_place)                                     # three tokens
        refused(big, 1000, in_place=in_place)                                   # three pages
        refused([10 ** 9, 0, 0, 0, 0, 0], 10, in_place=in_place)
        refused([2 ** 31 - 1] * 6, 1 << 20, in_place=in_place)
        refused(good, 10, kv=np.array([5, -1, 0, 0, 0, 0], np.int32), in_place=in_place)
        refused(good, 10, kv=np.array([2 ** 31 - 1, 0, 0, 0, 0, 0], np.int32), in_place=in_place)
        refused([s.max_pages * 16 + 1, 0, 0, 0, 0, 0], 4000, kv=np.zeros(6, np.int32), in_place=in_place)
        for ring in ((-1, 3), (s.n_pages, 3), (0, -1), (0, s.n_pages + 1), (0, s.n_pages)):
            refused(good, 10, ring=ring, in_place=in_place)


def test_page_numbers_that_name_no_page():
    s = State(2, 16, 0, spare=4, room=40)
    s.kv[:] = [20, 0]
    s.table[0, :2] = [s.n_pages, 1]
    s.free[:] = [0, 1, -4, 3]
    s.first = 1
    s.count = 3
    gq.gq_device_status()
    got = run(s, [13, 17], 30)
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    # request 0: positions 20 .. 31 in page 1, 32 in the ring's first (1); request 1: the ring's -4, then 3
    want = [1 * 16 + x % 16 for x in range(20, 32)] + [16] + [-1] * 16 + [3 * 16]
    assert list(got["slot"]) == want
    assert list(got["kv_len"]) == [33, 17] and list(got["sequence"]) == [0] * 13 + [1] * 17


def test_many_steps_in_place_keep_every_page():
    t = torch()
    g = np.random.default_rng(4)
    n, page, n_pages, max_pages, n_tokens = 40, 16, 300, 12, 200
    i32 = dict(dtype=t.int32, device="cuda")
    kv, ring = t.zeros(n, **i32), t.tensor([0, n_pages], **i32)
    free, table = t.randperm(n_pages).to(t.int32).cuda(), t.full((n, max_pages), -1, **i32)
    new, q_start = t.zeros(n, **i32), t.zeros(n + 1, **i32)
    slot = t.zeros(n_tokens, dtype=t.int64, device="cuda")
    seq, pos = t.zeros(n_tokens, **i32), t.zeros(n_tokens, **i32)

    def call():
        gq.gq_kv_plan(new, kv, ring, free, table, kv, q_start, ring, slot, pos, seq, n_pages, max_pages, page, n, n_tokens)

    call()  # nothing new: nothing changes
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        call()
    where = {}  # slot -> (request, position)
    gq.gq_device_status()
    for _ in range(60):
        old = kv.cpu().numpy()
        want = np.where(g.random(n) < 0.15, g.integers(0, 20, n), 1)
        want[(old > 150) | (g.random(n) < 0.05)] = -1
        new.copy_(t.from_numpy(want.astype(np.int32)))
        before = kv.clone()
        graph.replay()
        assert gq.gq_device_status() == gq.GQ_OK
        lens = kv.cpu().numpy()
        assert np.array_equal(lens, np.where(want < 0, 0, old + want))
        held = [int(p) for b in range(n) for p in table[b, :-(-int(lens[b]) // page)]]
        first, count = ring.tolist()
        ringed = [int(free[(first + i) % n_pages]) for i in range(count)]
        assert sorted(held + ringed) == list(range(n_pages))
        gone = {b for b in range(n) if want[b] < 0}
        where = {k: v for k, v in where.items() if v[0] not in gone}
        for a, b, c in zip(slot.tolist(), seq.tolist(), pos.tolist()):
            if a >= 0:
                assert a not in where, "a place in use"
                where[a] = (b, c)
        assert len(where) == lens.sum()
        del before


def test_the_lists_lead_the_cache():
    """Append and attention over planned lists, in a padded batch, against the same tokens in one contiguous request each."""
    t = torch()
    hk, hq, d, page, n_pages, max_pages, n = 2, 4, 64, 16, 40, 8, 3
    g = t.Generator(device="cuda").manual_seed(0)
    i32 = dict(dtype=t.int32, device="cuda")
    kv, ring, table = t.zeros(n, **i32), t.tensor([7, n_pages], **i32), t.full((n, max_pages), -1, **i32)
    free, q_start = t.randperm(n_pages).to(t.int32).cuda(), t.zeros(n + 1, **i32)
    cache = t.zeros(gq.gq_kv_cache_bytes(n_pages, page, hk, d), dtype=t.uint8, device="cuda")
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(hq, hk, d), dtype=t.uint8, device="cuda")
    slot = t.zeros(64, dtype=t.int64, device="cuda")
    seq, pos = t.zeros(64, **i32), t.zeros(64, **i32)
    kept = {b: [] for b in range(n)}
    gq.gq_device_status()
    for new in ([30, 1, 0], [1, 20, 17], [1, 1, 1], [-1, 1, 1], [40, 1, 1]):
        gq.gq_kv_plan(t.tensor(new, **i32), kv, ring, free, table, kv, q_start, ring, slot, pos, seq, n_pages, max_pages, page, n, 64)
        q, k, v = (t.randn(64, h * d, generator=g, device="cuda") for h in (hq, hk, hk))
        out = t.full((64, hq * d), 5.5, device="cuda")
        sizes = (n_pages, max_pages, page, hk, d, n, 64)
        gq.gq_kv_append_q8_0(k, hk * d, v, hk * d, 0, cache, table, kv, q_start, *sizes)
        gq.gq_kv_attention_q8_0(q, hq * d, cache, table, kv, q_start, out, hq * d, 0, d ** -0.5, 0.0, 0, ws, ws.numel(), hq, *sizes)
        total = int(q_start[n])
        assert bool((out[total:] == 5.5).all())
        for b in range(n):
            if new[b] < 0:
                kept[b] = []
            rows = [r for r in range(total) if int(seq[r]) == b]
            assert [int(pos[r]) for r in rows] == list(range(len(kept[b]), len(kept[b]) + len(rows)))
            kept[b] += [(k[r], v[r]) for r in rows]
            if not rows:
                continue
            kk = t.stack([x for x, _ in kept[b]]).view(-1, hk, d).double()
            vv = t.stack([x for _, x in kept[b]]).view(-1, hk, d).double()
            for r in rows:
                m = int(pos[r]) + 1
                s = t.einsum("hgd,nhd->hgn", q[r].view(hk, hq // hk, d).double(), kk[:m]) * d ** -0.5
                ref = t.einsum("hgn,nhd->hgd", s.softmax(-1), vv[:m]).reshape(-1)
                # codes of 8 bits: a key or value is off by 2^-8 of its block's largest (about 3), a score of 64 terms by
                # some 0.03, a result by that much of values of about 1, and its own 2^-8 of 3
                assert float((out[r] - ref).abs().max()) < 0.1
    assert gq.gq_device_status() == gq.GQ_OK
