"""Host-side checks of the workspace sizes of adapters and sampling (no GPU needed): a workspace of the largest batch
serves every smaller one."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
from block_quantized_matvec_gq_gb300 import build as gqbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    gqbuild.build()
    return gq.lib()


def counts(most):
    """1 .. 2000, where the divisions change most, and some of all sizes beyond, each with its neighbours."""
    far = np.unique(np.geomspace(2000, most - 1, 300).astype(np.int64))
    return [n for n in sorted({*range(1, 2001), *(int(x + d) for x in far for d in (-1, 0, 1))}) if n <= most]


@pytest.mark.parametrize("rank,K", [(8, 32), (16, 256), (16, 5376), (64, 4096), (128, 21504), (40, 100000), (16, 1 << 24)])
def test_adapters_of_fewer_tokens(rank, K):
    sizes = [gq.gq_lora_workspace_bytes(rank, K, m) for m in counts(1 << 28)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("M", [1, 8, 9, 300, 5000])
def test_adapters_of_smaller_ranks_and_rows(M):
    for K in (32, 4096, 20000):
        sizes = [gq.gq_lora_workspace_bytes(r, K, M) for r in range(8, gq.GQ_MAX_LORA_RANK + 1, 8)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    sizes = [gq.gq_lora_workspace_bytes(16, K, M) for K in range(32, 40000, 32)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("vocab", [1, 100, 4089, 4090, 8000, 8177, 8185, 12281, 32000, 65537, 262144, gq.GQ_MAX_VOCAB - 7, gq.GQ_MAX_VOCAB])
def test_sampling_of_fewer_rows(vocab):
    sizes = [gq.gq_sample_workspace_bytes(vocab, n) for n in counts(gq.GQ_MAX_SAMPLE_ROWS)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
