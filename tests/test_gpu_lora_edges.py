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


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("M,prompts", [(5, False), (40, True)])
def test_finite_numbers_beyond_the_largest_of_16_bits(M, prompts, typ):
    """3.4e38 lies between the largest bf16 (3.3895e38) and the largest f32: an activation, and a number of A x."""
    c = Case(M, 64, 36, 8, 2, [0, 1] if prompts else np.arange(M) % 3 - 1, runs([M // 2, M - M // 2]) if prompts else None, typ, False)
    c.x[:, 5] = np.float32(3.4e38) * np.where(np.arange(M) % 2, 1, -1).astype(np.float32)
    c.x[1, 5] = 1.0
    c.A[:, 3, 5] = 1.0
    c.B *= 2.0 ** -12
    c.scale[:] = 1.0
    assert np.all(np.isfinite(c.check()))


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("M,prompts", [(5, False), (40, True)])
def test_infinite_activations_give_no_finite_sums(M, prompts, typ):
    c = Case(M, 64, 36, 8, 2, [0, 1] if prompts else np.zeros(M, int), runs([M // 2, M - M // 2]) if prompts else None, typ, False)
    c.x[1, 5], c.x[2, 40] = np.inf, -np.inf
    got = c.run()
    bad = np.isin(np.arange(M), (1, 2))
    assert not np.any(np.isfinite(got[bad])) and np.all(np.isfinite(got[~bad]))


def bound_of(c):
    """Error bounds per element: the interface's three terms, the last with every activation, product and sum on the way
    cut by as much as 2^-126."""
    a, b = np.abs(c.A.double().cpu().numpy()), np.abs(c.B.double().cpu().numpy())
    y, bound, _ = c.reference()
    for i, ad in enumerate(c.of()):
        if ad >= 0:
            s, v = float(c.scale[ad]), a[ad] @ np.abs(c.x[i].astype(np.float64))
            if c.typ == "f16":
                bound[i] += 2.0 ** -38 * s * b[ad].sum(-1) * v.max()
            bound[i] += 2.0 ** -126 * (s * (b[ad] @ (a[ad].sum(-1) + 2 * c.K + 2)) + 2 * c.rank + 2)
    return y, bound


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("M,prompts", [(6, False), (40, True)])
def test_small_numbers_of_a_x_beside_large_ones(M, prompts, typ):
    """Number 0 of A x is 2^30 times number 3, and the first half of the rows of B takes number 3 alone."""
    c = Case(M, 64, 36, 8, 2, [0, 1] if prompts else np.arange(M) % 2, runs([M // 2, M - M // 2]) if prompts else None, typ, False)
    c.x[:, :32] *= np.float32(2.0 ** 15)
    c.x[:, 32:] *= np.float32(2.0 ** -15)
    c.A[:, 3, :32] = 0.0
    c.B[:, :18, :3] = 0.0
    c.B[:, :18, 4:] = 0.0
    c.y0[:, :18] = 0.0
    y, bound = bound_of(c)
    assert np.all(np.abs(c.run() - y) <= bound)


@pytest.mark.parametrize("f", [2.0 ** -110, 2.0 ** -122, 2.0 ** -130, 2.0 ** -140])
@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("M,prompts", [(6, False), (40, True)])
def test_activations_next_to_the_smallest(M, prompts, typ, f):
    c = Case(M, 64, 36, 8, 2, [0, 1] if prompts else np.arange(M) % 2, runs([M // 2, M - M // 2]) if prompts else None, typ, False)
    c.x = (c.x.astype(np.float64) * f).astype(np.float32)
    c.y0[:] = 0.0
    y, bound = bound_of(c)
    assert np.all(np.abs(c.run() - y) <= bound)
