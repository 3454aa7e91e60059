"""Sampling where its contract is sharpest: rows that a cluster of CTAs searches, most of which have nothing to read.

The reference and its tolerance are those of test_gpu_sample."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
from gpu_util import dev, torch
from test_gpu_sample import check, logits, sample, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [2100, 4300, 9001])
def test_searched_rows_of_which_most_ctas_read_nothing(vocab):
    """Flat rows with a min_p: the weight that it keeps is put together from all CTAs of the cluster, and in short rows
    the first of them is there at once.  The same again and again."""
    g = np.random.default_rng(vocab)
    n = 96
    x = dev(logits(g, n, vocab, False).astype(np.float32))
    s = dict(m=g.choice([0.15, 0.3, 0.6], n), p=g.choice([1.0, 0.8], n), k=g.choice([0, vocab - 7], n), u=g.random(n))
    token, prob = check(x, "f32", **s)
    for _ in range(50):
        again = sample(x, "f32", **s)
        assert np.array_equal(again[0], token) and np.array_equal(again[1], prob)


def test_smaller_calls_in_the_workspace_of_the_largest():
    """Sizes on both sides of where the slices change; the workspace ends with the bytes asked for."""
    t = torch()
    g = np.random.default_rng(3)
    vocab, most = 8000, 200
    size = gq.gq_sample_workspace_bytes(vocab, most)
    guarded_ws = t.full((size + 4096,), 0x5A, dtype=t.uint8, device="cuda")
    for n in (200, 153, 152, 151, 150, 9, 1):
        x, s = logits(g, n, vocab, n % 2 == 0), settings(g, n, vocab)
        got, want = sample(x, "f32", **s, ws=guarded_ws[:size]), sample(x, "f32", **s)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        assert bool((guarded_ws[size:] == 0x5A).all())


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab,ties", [(40, 3), (5000, 3), (70001, 3), (5000, 4000), (70001, 30000)])
@pytest.mark.parametrize("m", [1.0, 1.5, 3e38, float("inf")])
def test_a_min_p_of_one_or_more_keeps_what_ties_with_the_largest(vocab, ties, typ, m):
    """Few ties, which the lists settle, and many, which are searched; a quarter of an octave lies below them."""
    g = np.random.default_rng(ties)
    x = np.full((4, vocab), 2.0) - 0.25 * g.integers(1, 9, (4, vocab))
    at = np.sort(np.stack([g.choice(vocab, ties, replace=False) for _ in range(4)]), -1)
    np.put_along_axis(x, at, 2.0, -1)
    u = np.array([0.0, 0.4, 0.7, 0.9999], np.float32)
    token, prob = sample(x, typ, m=m, u=u)
    want = [at[r][int(np.floor(float(u[r]) * ties))] for r in range(4)]
    assert token.tolist() == want
    # a quotient of whole numbers brought to 24 bits each: three roundings
    assert np.all(np.abs(prob.astype(np.float64) * ties - 1) <= 3 * 2.0 ** -24 * (1 + 2.0 ** -20))


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("u", [1.0, 2.0, float("inf")])
def test_a_u_of_one_gives_the_last_kept_that_has_weight(u, typ):
    g = np.random.default_rng(4)
    low = {"f32": -3.4028235e38, "f16": -65504.0, "bf16": -3.3895314e38}[typ]
    for vocab in (2, 300, 5000, 70001):
        x = np.full((5, vocab), low)                        # masked with the lowest value
        last = np.zeros(5, int)
        x[0, :2] = 0.0, -40.0                               # 57 octaves below: no weight
        x[1, :2] = 0.0, -20.0                               # 28 octaves below
        last[1] = 1
        some = min(vocab - 1, 3000)
        x[2, g.permutation(vocab)[:some]] = 0.0             # as many equal ones, nothing else
        last[2] = np.flatnonzero(x[2] == 0.0)[-1]
        x[3] = 1.5                                          # all equal
        last[3] = vocab - 1
        at = g.choice(vocab, 2, replace=False)
        x[4, at] = 0.0, -10.0
        last[4] = at[1]
        token, _ = sample(x, typ, u=u)
        assert token.tolist() == last.tolist(), vocab
        token, _ = sample(x, typ, u=u, T=[1.0, 0.4, 1.0, 1.0, 0.1], k=[0, 2, some, vocab // 2 + 1, 0])
        assert token.tolist() == [0, 0, last[2], vocab // 2, at[0]], vocab
