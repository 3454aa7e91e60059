"""Sampling where its contract is sharpest: rows that a cluster of CTAs searches, most of which have nothing to read.

The reference and its tolerance are those of test_gpu_sample."""

import numpy as np
import pytest

from gpu_util import dev
from test_gpu_sample import check, logits, sample

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
