"""Host-side checks of the paged cache's C entry points (no GPU needed), and
of the plain record layout that the GPU tests compare with."""

import ctypes

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import kv_plain as kp
from block_quantized_matvec_gq_gb300 import build as gqbuild

A = 1 << 20          # aligned, never dereferenced
U = (1 << 20) + 4    # 4-byte aligned only


@pytest.fixture(scope="module", autouse=True)
def lib():
    gqbuild.build()
    return gq.lib()


def call(name, good, **kw):
    args = dict(good, **kw)
    return getattr(gq.lib(), name)(*args.values(), None)


SIZES = dict(n_pages=4, max_pages=4, page=16, kv_heads=2, dim=64, n_seq=1, n_tokens=3)
APPEND = dict(K=A, ldk=128, V=A, ldv=128, type=0, cache=A, table=A, kv_len=A, q_start=A, **SIZES)
READ = dict(cache=A, table=A, kv_len=A, q_start=A, K=A, ldk=128, V=A, ldv=128, type=0, **SIZES)
ATTEND = dict(Q=A, ldq=256, cache=A, table=A, kv_len=A, q_start=A, O=A, ldo=256, type=0, scale=ctypes.c_float(0.1),
              softcap=ctypes.c_float(0.0), window=0, ws=A, ws_bytes=1 << 40, heads=4, **SIZES)
ENTRIES = [("gq_kv_append_q8_0", APPEND), ("gq_kv_read_q8_0", READ), ("gq_kv_attention_q8_0", ATTEND)]


@pytest.mark.parametrize("name,good", ENTRIES)
def test_refusals(name, good):
    for p in ("K", "V", "Q", "O", "cache"):
        if p in good:
            assert call(name, good, **{p: None}) == gq.GQ_ERR_NULL, p
            assert call(name, good, **{p: U}) == gq.GQ_ERR_ALIGN, p
    for p in ("table", "kv_len", "q_start"):
        assert call(name, good, **{p: None}) == gq.GQ_ERR_NULL, p
        assert call(name, good, **{p: A + 2}) == gq.GQ_ERR_ALIGN, p
    for p in ("ldk", "ldv", "ldq", "ldo"):
        if p in good:
            assert call(name, good, **{p: good[p] - 4}) == gq.GQ_ERR_SHAPE, p
            assert call(name, good, **{p: good[p] + 2}) == gq.GQ_ERR_ALIGN, p          # 8 bytes off in f32
            assert call(name, good, type=1, **{p: good[p] + 4}) == gq.GQ_ERR_ALIGN, p  # and in f16
    assert call(name, good, type=3) == gq.GQ_ERR_FORMAT
    assert call(name, good, type=-1) == gq.GQ_ERR_FORMAT
    for p, bad in (("n_pages", 0), ("max_pages", 0), ("page", 0), ("page", 24), ("page", 4112), ("kv_heads", 0), ("dim", 32),
                   ("dim", 96), ("dim", 0), ("dim", 512), ("n_seq", 0), ("n_tokens", -1), ("n_tokens", (1 << 28) + 1),
                   ("max_pages", 1 << 27), ("kv_heads", 1 << 20)):
        assert call(name, good, **{p: bad}) == gq.GQ_ERR_SHAPE, (p, bad)
    assert call(name, good, n_tokens=0) == gq.GQ_OK  # nothing to do, nothing launched


def test_attention_refusals():
    f = ctypes.c_float
    name = "gq_kv_attention_q8_0"
    assert call(name, ATTEND, ws=None) == gq.GQ_ERR_WORKSPACE
    need = gq.gq_kv_attention_workspace_bytes(4, 2, 64)
    assert need > 0
    assert call(name, ATTEND, ws_bytes=need - 1) == gq.GQ_ERR_WORKSPACE
    assert call(name, ATTEND, ws=U) == gq.GQ_ERR_ALIGN
    assert call(name, ATTEND, window=-1) == gq.GQ_ERR_SHAPE
    assert call(name, ATTEND, heads=3) == gq.GQ_ERR_SHAPE
    assert call(name, ATTEND, heads=0) == gq.GQ_ERR_SHAPE
    for bad in (float("nan"), float("inf")):
        assert call(name, ATTEND, scale=f(bad)) == gq.GQ_ERR_SHAPE
        assert call(name, ATTEND, softcap=f(bad)) == gq.GQ_ERR_SHAPE


def test_sizes():
    assert gq.gq_kv_cache_bytes(3, 64, 8, 128) == 3 * 8 * 4 * 34 * 128
    assert gq.gq_kv_cache_bytes(1 << 20, 4096, 8, 256) == (1 << 20) * 8 * 256 * 34 * 256  # beyond 32 bits
    for bad in ((0, 16, 1, 64), (1, 8, 1, 64), (1, 16, 0, 64), (1, 16, 1, 80)):
        assert gq.gq_kv_cache_bytes(*bad) == 0
    for bad in ((3, 2, 64), (2, 0, 64), (1, 2, 64), (4, 2, 100)):
        assert gq.gq_kv_attention_workspace_bytes(*bad) == 0


def test_the_binding_refuses_what_it_cannot_pass():
    import torch
    x = torch.zeros(3, 128)
    with pytest.raises(ValueError):
        gq.gq_kv_append_q8_0(x, 128, x, 128, 0, x, x, x, x, 4, 4, 16, 2, 64, 1, 3)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_layout_uses_every_byte_of_a_record_once(dim):
    kc, ks, vc, vs = kp.layout(dim)
    used = np.concatenate([kc.ravel(), vc.ravel(), ks.ravel(), ks.ravel() + 1, vs.ravel(), vs.ravel() + 1])
    assert np.array_equal(np.sort(used), np.arange(34 * dim))


def test_plain_write_and_read_are_inverse():
    rng = np.random.default_rng(1)
    batch = kp.make([21, 5], [21, 5], 2, 64, 16, rng)
    want = []
    for b in range(2):
        for p in batch.positions(b):
            k, v = rng.standard_normal((2, 2, 64)).astype(np.float32)
            kp.write(batch, b, p, k, v)
            want.append([kp.quantise(x) for x in (k, v)])
    got = [kp.values(batch, b, batch.positions(b)) for b in range(2)]
    for i in range(2):
        have = np.concatenate([g[i] for g in got])
        for n, w in enumerate(want):
            code, d = w[i]
            assert np.array_equal(have[n], code * np.repeat(d.astype(np.float64), 32, -1))
    x = rng.standard_normal((5, 96)).astype(np.float32)
    code, d = kp.quantise(x)
    assert np.abs(code * np.repeat(d.astype(np.float64), 32, -1) - x).max() <= 0.51 * d.astype(np.float64).max()
