"""The example block: prompt chunks and single tokens through one cache."""

import os
import sys

import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_example_runs_and_agrees_with_the_cache_read_back():
    import attention_step
    t = torch()
    y, err = attention_step.main()
    assert y.shape == (81, 1024) and bool(t.isfinite(y).all())
    # torch's f32 products against the kernel's: both within a few roundings of 2^-24 per term
    assert err < 1e-5
