"""Sampling against the definition in 64 bits.

Which token is right is exact except where a target lies within rounding of a
running weight.  Weights are within 2^-23 of themselves and 2^-42 of the
largest: a running weight is off by at most 2^-23 of the total, plus 2^-42 times
the row's length of the largest (below 2^-23 up to 2^19 elements), a ratio of two
of them by twice their sum: 2^-21.  `allowed` takes top_p, min_p and u that much
to either side and collects every token that some choice gives; prob within the
same 2^-21 of one of them, its own rounding (2^-22, three roundings), and the
2^-42 of the largest weight that a weight may be off by itself."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
from gpu_util import dev, torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": gq.GQ_TYPE_F32, "f16": gq.GQ_TYPE_F16, "bf16": gq.GQ_TYPE_BF16}
OFF = 2.0 ** -21


def tt(typ):
    return {"f32": torch().float32, "f16": torch().float16, "bf16": torch().bfloat16}[typ]


def allowed(row, T, k, p, m, u):
    """{token: probs} that the definition gives for settings within OFF of these; row in 64 bits."""
    row = np.where(np.isnan(row), -np.inf, row)
    order = np.lexsort((np.arange(len(row)), -row))
    order = order[row[order] > -np.inf]
    if not len(order) or np.isnan([T, p, m]).any():
        return {-1: [0.0]}
    if T <= 0:
        return {int(order[0]): [1.0]}
    if k > 0:
        order = order[:k]
    top = row[order[0]]
    with np.errstate(invalid="ignore"):
        far = 0.0 if top == np.inf else np.exp((row[order] - top) / max(T, 2.0 ** -100))
        w = np.where(row[order] == top, 1.0, far)
    F = np.cumsum(w)
    u = 0.0 if np.isnan(u) else min(max(u, 0.0), 1.0)
    kept = set()
    for e in (1 - OFF, 1.0, 1 + OFF):
        n_p = len(w) if p >= 1 else 1 + int(np.searchsorted(F, p * e * F[-1])) if p > 0 else 1
        n_m = max(1, int(np.count_nonzero(w >= m * e))) if 0 < m < 1 else max(1, int(np.count_nonzero(w >= 1))) if m >= 1 else len(w)
        kept.add(min(n_p, n_m, len(w)))
    got = {}
    for n in kept:
        z = F[n - 1]
        lo = int(np.searchsorted(F[:n], (u - OFF) * z, side="right"))
        hi = int(np.searchsorted(F[:n], (u + OFF) * z, side="right"))
        last = int(np.max(np.nonzero(w[:n])))
        for j in range(min(lo, last), min(hi, last) + 1):
            got.setdefault(int(order[j]), []).append(w[j] / z)
    return got


def sample(x, typ, T=None, k=None, p=None, m=None, u=0.5, with_prob=True, ws=None):
    """x: float array [n][vocab], or a device tensor with any row stride."""
    t = torch()
    x = dev(np.asarray(x, np.float32)).to(tt(typ)) if isinstance(x, np.ndarray) else x
    n, vocab = x.shape
    arr = lambda v, d: None if v is None else dev(np.broadcast_to(np.asarray(v, d), (n,)).copy())  # noqa: E731
    token = t.full((n + 2,), -77, dtype=t.int32, device="cuda")
    prob = t.full((n + 2,), -77.0, device="cuda")
    if ws is None:
        ws = t.full((gq.gq_sample_workspace_bytes(vocab, n),), 0xA5, dtype=t.uint8, device="cuda")
    gq.gq_sample(x, x.stride(0), TYPES[typ], arr(T, np.float32), arr(k, np.int32), arr(p, np.float32), arr(m, np.float32),
                 arr(u, np.float32), token, prob if with_prob else None, ws, ws.numel(), vocab, n)
    token, prob = token.cpu().numpy(), prob.cpu().numpy()
    assert np.all(token[n:] == -77) and np.all(prob[n:] == -77), "written outside"
    return token[:n], prob[:n]


def check(x, typ, T=1.0, k=0, p=1.0, m=0.0, u=0.5):
    t = torch()
    x = dev(np.asarray(x, np.float32)).to(tt(typ)) if isinstance(x, np.ndarray) else x
    n = x.shape[0]
    per = [np.broadcast_to(np.asarray(v, d), (n,)) for v, d in ((T, np.float32), (k, np.int32), (p, np.float32), (m, np.float32), (u, np.float32))]
    token, prob = sample(x, typ, *per)
    rows = x.double().cpu().numpy()
    for r in range(n):
        ok = allowed(rows[r], *(float(v[r]) if i != 1 else int(v[r]) for i, v in enumerate(per)))
        what = (r, int(token[r]), float(prob[r]), [v[r] for v in per], dict(list(ok.items())[:4]))
        assert int(token[r]) in ok, what
        # a probability is at most 1, so 2^-42 of the largest weight is at most 2^-42 here
        assert any(abs(prob[r] - q) <= (2 * OFF + 2.0 ** -22) * q + 2.0 ** -42 for q in ok[int(token[r])]), what
    return token, prob


def settings(g, n, vocab):
    return dict(T=g.choice([0.0, 0.3, 0.8, 1.0, 1.3, 4.0], n), k=g.choice([0, 0, 1, 7, 50, 1000, vocab - 1, vocab, 1 << 30, -3], n),
                p=g.choice([1.0, 1.5, 0.0, -1.0, 0.1, 0.5, 0.9, 0.999], n), m=g.choice([0.0, -1.0, 0.001, 0.1, 0.9, 1.0, 2.0], n),
                u=g.choice([0.0, 0.999999, 1.0, -1.0, *g.random(4)], n))


def logits(g, n, vocab, sharp):
    """sharp: a language model's tail; else noise, where nearly every token keeps some weight."""
    return g.exponential(1.5, (n, vocab)) - 4.0 if sharp else g.standard_normal((n, vocab)) * 0.3


@pytest.mark.parametrize("sharp", [True, False])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n,vocab", [(3, 1), (4, 2), (9, 31), (40, 1000), (7, 4095), (33, 4097), (12, 16390), (21, 70001), (5, 262144)])
def test_settings(n, vocab, typ, sharp):
    g = np.random.default_rng(vocab + sharp)
    check(logits(g, n, vocab, sharp), typ, **settings(g, n, vocab))


def test_a_large_batch():
    """Enough rows for the long slices; every limit alone, at the flat end."""
    g = np.random.default_rng(5)
    n, vocab = 180, 40000
    check(logits(g, n, vocab, True), "f32", **settings(g, n, vocab))
    check(logits(g, n, vocab, False), "bf16", **settings(g, n, vocab))


@pytest.mark.parametrize("limit", [dict(k=3000), dict(k=30000), dict(p=0.3), dict(p=0.97), dict(m=0.2), dict(T=50.0), dict(T=float("inf")), {}])
def test_one_limit_over_flat_rows(limit):
    g = np.random.default_rng(6)
    u = np.array([0.0, 1e-7, 0.1, 0.37, 0.5, 0.77, 0.9, 0.99999])
    check(logits(g, 8, 50021, False), "f32", u=u, **limit)


def test_the_same_whatever_the_batch():
    """One row alone goes through short slices, in a batch through long ones."""
    g = np.random.default_rng(7)
    x, s = logits(g, 200, 30011, True), settings(g, 200, 30011)
    x[::3] *= 0.2
    token, prob = sample(x, "f32", **s)
    for r in range(0, 200, 9):
        one = sample(x[r:r + 1], "f32", **{a: v[r] for a, v in s.items()})
        # sums of slices are cut at 2^-43 of the slice's largest: prob to the last bit or two
        assert one[0][0] == token[r] and abs(one[1][0] - prob[r]) <= 2.0 ** -22 * prob[r]


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("vocab", [5, 3000, 40000, 300007])
def test_equal_logits_go_by_index(vocab, typ):
    """All weights equal: the token is the index at which (i + 1) / V first exceeds u."""
    u = np.array([0.0, 0.25, 0.5, 0.8125, 0.9999], np.float32)
    x = np.full((5, vocab), 3.25)
    token, prob = sample(x, typ, u=u, T=0.7)
    assert np.array_equal(token, np.floor(u.astype(np.float64) * vocab).astype(int))
    assert np.all(np.abs(prob * vocab - 1) < 2.0 ** -21)
    k = max(1, vocab // 3)
    token, prob = sample(x, typ, u=u, k=k)
    assert np.array_equal(token, np.floor(u.astype(np.float64) * k).astype(int))
    token, _ = sample(x, typ, T=0.0)
    assert np.all(token == 0)


def test_many_ties_at_a_few_values():
    g = np.random.default_rng(8)
    x = g.integers(0, 4, (24, 33000)).astype(np.float64)
    check(x, "bf16", u=g.random(24), k=g.choice([0, 1, 5000, 20000], 24), p=g.choice([1.0, 0.5, 0.95], 24))


def test_masked_rows():
    g = np.random.default_rng(9)
    for typ, low in (("f32", -3.4028235e38), ("f16", -65504.0), ("bf16", -3.3895314e38)):
        x = logits(g, 8, 9000, True)
        x[0] = -np.inf                     # nothing allowed
        x[1] = np.nan
        x[2, 10:] = -np.inf
        x[3, :] = -np.inf
        x[3, 8765] = -2.0                  # one allowed
        x[4, 5:] = low                     # masked with the lowest value
        x[5] = low                         # all of them
        x[6, ::2] = np.nan
        x[7, 1:] = -np.inf
        x[7, 0] = low
        token, prob = check(x, typ, u=g.random(8), p=[1, 1, 0.9, 0.9, 1, 1, 0.9, 1.0])
        assert token[0] == -1 == token[1] and prob[0] == 0 == prob[1] and token[3] == 8765 and prob[3] == 1


@pytest.mark.parametrize("vocab", [100, 20000])
def test_infinities_share_the_weight(vocab):
    x = np.zeros((6, vocab))
    x[:, [7, 50, 99]] = np.inf
    token, prob = check(x, "f32", u=[0.0, 0.3, 0.34, 0.7, 0.99, 0.5], T=[1, 1, 2, 1, float("inf"), 0.0])
    assert list(token[:4]) == [7, 7, 50, 99]


def test_zero_and_minus_zero_are_equal():
    x = np.zeros((4, 300))
    x[:, ::2] = -0.0
    token, _ = sample(x, "f32", u=[0.0, 0.25, 0.5, 0.99], k=[0, 100, 2, 3])
    assert list(token) == [0, 25, 1, 2]


def test_extreme_temperatures_and_logits():
    g = np.random.default_rng(10)
    x = logits(g, 10, 5000, True)
    x[5:] *= 1e30
    x[7] = 1e30 * (1 + np.arange(5000) % 3 * 2.0 ** -23)      # neighbours a unit apart, T about as large
    T = [1e-38, 1e-20, 1e-5, 1e5, 1e38, 1.0, 1e30, 1e23, 1e-30, 3e38]
    check(x, "f32", T=T, u=g.random(10), p=[1, 0.9] * 5)


def test_bad_settings_are_refused_row_by_row():
    gq.gq_device_status()
    x = np.tile(np.arange(50.0), (5, 1))
    nan = float("nan")
    token, prob = sample(x, "f32", T=[nan, 1, 1, 1, 0], p=[1, nan, 1, 1, 1], m=[0, 0, nan, 0, 0], u=[0.5, 0.5, 0.5, nan, nan])
    assert list(token) == [-1, -1, -1, 49, 49] and list(prob[:3]) == [0, 0, 0]
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    assert gq.gq_device_status() == gq.GQ_OK


def test_defaults_without_arrays():
    g = np.random.default_rng(11)
    x = logits(g, 6, 777, True)
    u = g.random(6).astype(np.float32)
    a = sample(x, "f32", u=u)
    b = sample(x, "f32", T=1.0, k=0, p=1.0, m=0.0, u=u, with_prob=False)
    assert np.array_equal(a[0], b[0])


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1003), (3, 1024), (5, 1001), (7, 1007)])
def test_rows_that_begin_anywhere(offset, stride, typ):
    """Neighbouring elements are far above every logit: reading one would show."""
    t = torch()
    g = np.random.default_rng(offset)
    flat = t.full((offset + 4 * stride + 16,), 100.0, dtype=tt(typ), device="cuda")
    x = flat[offset:offset + 4 * stride].view(4, stride)[:, :1000]
    x.copy_(dev(logits(g, 4, 1000, True).astype(np.float32)))
    check(x, typ, u=g.random(4), k=[0, 1, 20, 0])


def test_captured_and_replayed_with_other_logits_and_settings():
    t = torch()
    g = np.random.default_rng(12)
    n, vocab = 6, 20011
    ws = t.zeros(gq.gq_sample_workspace_bytes(vocab, n), dtype=t.uint8, device="cuda")
    x, T, u = t.zeros(n, vocab, device="cuda"), t.ones(n, device="cuda"), t.zeros(n, device="cuda")
    k = t.zeros(n, dtype=t.int32, device="cuda")
    token, prob = t.zeros(n, dtype=t.int32, device="cuda"), t.zeros(n, device="cuda")

    def call():
        gq.gq_sample(x, vocab, gq.GQ_TYPE_F32, T, k, None, None, u, token, prob, ws, ws.numel(), vocab, n)

    call()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        call()
    for sharp in (True, False, True):
        new, s = logits(g, n, vocab, sharp).astype(np.float32), settings(g, n, vocab)
        x.copy_(dev(new))
        for a, b in ((T, s["T"]), (u, s["u"]), (k, s["k"])):
            a.copy_(t.from_numpy(np.asarray(b)))
        graph.replay()
        want = sample(new, "f32", T=s["T"], k=s["k"], u=s["u"])
        assert np.array_equal(token.cpu().numpy(), want[0]) and np.array_equal(prob.cpu().numpy(), want[1])


def test_two_streams_with_a_workspace_each():
    t = torch()
    g = np.random.default_rng(13)
    xs = [dev(logits(g, 20, 30000, s).astype(np.float32)) for s in (True, False)]
    u = g.random(20)
    alone = [sample(x, "f32", u=u, p=0.9) for x in xs]
    streams = [t.cuda.Stream() for _ in xs]
    t.cuda.synchronize()
    for _ in range(4):
        for i, x in enumerate(xs):
            with t.cuda.stream(streams[i]):
                got = sample(x, "f32", u=u, p=0.9)
            assert np.array_equal(got[0], alone[i][0]) and np.array_equal(got[1], alone[i][1])


def test_one_workspace_for_calls_of_any_size():
    t = torch()
    g = np.random.default_rng(15)
    ws = t.zeros(max(gq.gq_sample_workspace_bytes(*s) for s in ((60000, 30), (300, 700), (200000, 1))), dtype=t.uint8, device="cuda")
    for vocab, n in ((60000, 30), (300, 700), (200000, 1), (300, 2), (60000, 29), (5, 1)):
        x, s = logits(g, n, vocab, vocab % 1000 == 0), settings(g, n, vocab)
        got, want = sample(x, "f32", **s, ws=ws), sample(x, "f32", **s)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("limit", [dict(m=0.3), dict(m=0.02, p=0.9), dict(p=0.2), dict(p=0.5), {}])
def test_a_top_k_beyond_the_list(limit):
    """Whether the list settles it depends on the other limits; sharp and flat rows."""
    g = np.random.default_rng(16)
    n, vocab = 30, 50000
    x = logits(g, n, vocab, True) * np.linspace(0.3, 2.0, n)[:, None]
    check(x, "f32", u=g.random(n), k=g.choice([1500, 4000, 20000, 49999], n), **limit)


def test_the_largest_vocabulary():
    g = np.random.default_rng(14)
    x = logits(g, 2, gq.GQ_MAX_VOCAB, True)
    x[1] = 0.0
    token, prob = check(x[:1], "f32", u=0.6, p=0.95)
    token, prob = sample(x[1:], "f32", u=0.75)
    assert token[0] == gq.GQ_MAX_VOCAB * 3 // 4


def test_frequencies_follow_the_probabilities():
    """A grid of u draws every token in proportion to its weight."""
    x = np.log(np.array([4.0, 1.0, 2.0, 1.0]))[None].repeat(800, 0)
    token, prob = sample(x, "f32", u=(np.arange(800) + 0.5) / 800)
    assert list(np.bincount(token, minlength=4)) == [400, 100, 200, 100]
    assert np.allclose(prob, np.array([0.5, 0.125, 0.25, 0.125])[token], rtol=2.0 ** -20)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("vocab", [2047, 2048, 2049, 4089, 4090])
def test_rows_about_as_long_as_the_list_or_a_slice(vocab, typ):
    g = np.random.default_rng(vocab)
    for sharp in (True, False):
        check(logits(g, 12, vocab, sharp), typ, **settings(g, 12, vocab))
    token, prob = sample(np.zeros((3, vocab)), typ, u=np.array([0.0, 0.5, 1.0]), k=vocab - 1)
    assert token.tolist() == [0, (vocab - 1) // 2, vocab - 2]
    assert np.all(np.abs(prob * (vocab - 1) - 1) < 2.0 ** -21)


def test_limits_that_fall_into_one_crowded_step_and_others_that_do_not():
    """Searched rows: thousands of equal logits where one of top_k, top_p and the draw ends, a smooth slope at the others."""
    g = np.random.default_rng(12)
    vocab = 60013
    x = np.tile(np.sort(g.standard_normal(vocab) * 0.4)[::-1], (9, 1))
    for r in range(9):
        a = [3000, 9000, 30000][r % 3]
        x[r, a:a + 5000] = x[r, a]
        x[r] = x[r, g.permutation(vocab)]
    k = np.repeat([0, 10000, 40000], 3)
    for p, m in ((1.0, 0.0), (0.2, 0.0), (0.7, 0.3), (0.999, 0.9)):
        check(x, "f32", k=k, p=p, m=m, u=g.random(9))
