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
