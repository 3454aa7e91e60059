"""Rows of a packed table by token id, bit for bit: every format and type, odd
sizes, strides, repeated, padded and bad ids."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import oracle
import synth
from gpu_util import dev, packed, torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": gq.GQ_TYPE_F32, "f16": gq.GQ_TYPE_F16, "bf16": gq.GQ_TYPE_BF16}


def tt(typ):
    return {"f32": torch().float32, "f16": torch().float16, "bf16": torch().bfloat16}[typ]


def table(fmt, rows, K, seed=0):
    W = synth.weights(fmt, rows, K, synth.stream(900 + fmt, seed))
    # the weights in 64 bits, exact but for Q4_K's difference and Q6_K's product, which f32 rounds once
    return packed(fmt, W, rows, K), oracle.dequant(fmt, W.reshape(-1), rows * K).reshape(rows, K).astype(np.float32)


def want(w, ids, scale, typ):
    """The documented roundings: f32 product, then the type."""
    t = torch()
    y = np.zeros((len(ids), w.shape[1]), np.float32)
    ok = (ids >= 0) & (ids < w.shape[0])
    y[ok] = w[ids[ok]] * np.float32(scale)
    return t.from_numpy(y).to(tt(typ))


def embed(fmt, Wp, ids, scale, typ, rows, K, pad=0, fill=-7.5):
    t = torch()
    y = t.full((len(ids) + 1, K + pad), fill, dtype=tt(typ), device="cuda")
    gq.gq_embed(fmt, Wp, dev(ids), scale, y[:, :K], y.stride(0), TYPES[typ], rows, K, len(ids))
    y = y.cpu()
    assert bool((y[len(ids)] == fill).all()) and bool((y[:, K:] == fill).all()), "written outside"
    return y[:len(ids), :K]


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("fmt,rows,K", [(0, 3, 32), (0, 50, 4128), (1, 7, 96), (1, 300, 5376), (2, 1, 256), (2, 77, 5376),
                                        (3, 1, 256), (3, 77, 5376)])
def test_rows(fmt, rows, K, typ):
    Wp, w = table(fmt, rows, K)
    ids = synth.stream(901, K).integers(0, rows, 41).astype(np.int32)
    ids[3] = ids[4] = ids[40]
    ids[5] = rows - 1
    for scale, pad, m in ((K ** 0.5, 0, 41), (-0.37, 8, 1), (1.0, 16, 2)):
        got = embed(fmt, Wp, ids[:m], scale, typ, rows, K, pad)
        assert torch().equal(got, want(w, ids[:m], scale, typ))


def test_many_tokens():
    Wp, w = table(1, 1000, 2048)
    ids = synth.stream(902, 0).integers(0, 1000, 20011).astype(np.int32)
    assert torch().equal(embed(1, Wp, ids, 3.25, "bf16", 1000, 2048), want(w, ids, 3.25, "bf16"))


def test_padding_and_bad_ids():
    Wp, w = table(0, 9, 64)
    gq.gq_device_status()
    ids = np.array([2, -1, 8, -2 ** 31, 0], np.int32)
    assert torch().equal(embed(0, Wp, ids, 2.0, "f32", 9, 64), want(w, ids, 2.0, "f32"))
    assert gq.gq_device_status() == gq.GQ_OK
    ids = np.array([2, 9, 8, 2 ** 31 - 1], np.int32)
    assert torch().equal(embed(0, Wp, ids, 2.0, "f32", 9, 64), want(w, ids, 2.0, "f32"))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    assert gq.gq_device_status() == gq.GQ_OK


def test_offsets_beyond_32_bits():
    """The last rows of a table of more than 4 GiB."""
    t = torch()
    rows, K = 1 << 20, 4096
    n = gq.gq_packed_bytes(1, rows, K)
    assert n > 1 << 32
    Wp = t.zeros(n, dtype=t.uint8, device="cuda")
    codes = t.randint(0, 256, (3, K), dtype=t.uint8, device="cuda")
    Wp[(rows - 3) * K:rows * K] = codes.flatten()
    d = t.rand(3, K // 32, device="cuda").half()
    Wp[rows * K + (rows - 3) * (K // 32) * 2:] = d.flatten().view(t.uint8)
    ids = np.array([rows - 1, rows - 3, rows - 2], np.int32)
    got = embed(1, Wp, ids, 1.0, "f32", rows, K)
    ref = (codes.float() - 128).view(3, K // 32, 32) * d.float()[..., None]
    assert t.equal(got, ref.view(3, K)[[2, 0, 1]].cpu())


def test_captured_with_other_ids_and_no_tokens():
    t = torch()
    Wp, w = table(2, 40, 512)
    ids, y = t.zeros(4, dtype=t.int32, device="cuda"), t.empty(4, 512, device="cuda")
    gq.gq_embed(2, Wp, None, 1.0, None, 512, 0, 40, 512, 0)
    gq.gq_embed(2, Wp, ids, 1.5, y, 512, 0, 40, 512, 4)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        gq.gq_embed(2, Wp, ids, 1.5, y, 512, 0, 40, 512, 4)
    for new in ([1, 2, 3, 39], [5, -1, 5, 0]):
        ids.copy_(t.tensor(new, dtype=t.int32))
        graph.replay()
        assert t.equal(y.cpu(), want(w, np.array(new), 1.5, "f32"))
