"""Adapters where their contract is sharpest.  The reference and its tolerance are those of test_gpu_lora."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
from gpu_util import torch
from test_gpu_lora import Case, runs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
def test_smaller_calls_in_the_workspace_of_the_largest(q8):
    """Decode batches and prompts of fewer tokens, whose sums have more slices; the workspace ends with the bytes asked for."""
    t = torch()
    K, rows, rank, most = 5376, 36, 16, 4096
    size = gq.gq_lora_workspace_bytes(rank, K, most)
    ws = t.full((size + 4096,), 0x5A, dtype=t.uint8, device="cuda")
    for M, prompts in ((520, True), (512, True), (512, False), (300, False), (64, True), (49, False), (48, False), (9, True), (1, False)):
        sequence = runs([M // 2, M - M // 2]) if prompts else None
        adapter = [1, 0] if prompts else np.arange(M) % 4 - 1
        c = Case(M, K, rows, rank, 3, adapter, sequence, "bf16", q8, seed=M)
        assert np.array_equal(c.check(ws=ws[:size]), c.run()), M
        assert bool((ws[size:] == 0x5A).all())
