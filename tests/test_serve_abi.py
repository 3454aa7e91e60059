"""Host-side checks (no GPU) of the entry points of a serving step: lists,
embedding rows, adapters and sampling refuse what they cannot compute before
any launch, and a call without work does nothing."""

import ctypes

import pytest

import block_quantized_matvec_gq_gb300 as gq
from block_quantized_matvec_gq_gb300 import build as gqbuild

A = 1 << 20          # aligned, never dereferenced
B = 1 << 21
U = (1 << 20) + 4    # 4-byte aligned only
F = ctypes.c_float
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    gqbuild.build()
    return gq.lib()


PLAN = dict(n_new=A, kv_in=A, ring_in=A, free=A, table=A, kv_len=A, q_start=A, ring=A, slot=A, position=A, sequence=A,
            n_pages=4, max_pages=4, page=16, n_seq=2, n_tokens=3)
EMBED = dict(format=1, W=A, ids=A, scale=F(1.0), Y=A, ldy=256, type=0, rows=10, K=256, M=2)
LORA = dict(A=A, B=A, type=2, scale=A, adapter=A, sequence=A, X=A, ldx=64, Y0=A, ldy0=32, Y=B, ldy=32, ws=A, ws_bytes=1 << 40,
            n_adapters=3, rank=16, rows=32, K=64, n_seq=2, M=5)
LORA8 = dict(A=A, B=A, type=2, scale=A, adapter=A, sequence=A, Xq=A, dx=A, Y0=A, ldy0=32, Y=B, ldy=32, ws=A, ws_bytes=1 << 40,
             n_adapters=3, rank=16, rows=32, K=64, n_seq=2, M=5)
SAMPLE = dict(logits=A, ldl=100, type=0, t=A, k=A, p=A, m=A, u=A, token=A, prob=A, ws=A, ws_bytes=1 << 40, vocab=100, n=3)


def call(name, good, **kw):
    assert set(kw) <= set(good)
    return getattr(gq.lib(), name)(*dict(good, **kw).values(), None)


def refuses(name, good, status, **bad):
    for arg, values in bad.items():
        for v in values:
            assert call(name, good, **{arg: v}) == status, (arg, v)


def test_plan():
    name = "gq_kv_plan"
    lists = ("n_new", "kv_in", "ring_in", "free", "table", "kv_len", "q_start", "ring")
    refuses(name, PLAN, gq.GQ_ERR_NULL, **{p: [None] for p in lists})
    refuses(name, PLAN, gq.GQ_ERR_ALIGN, **{p: [A + 2] for p in lists + ("position", "sequence")}, slot=[A + 4])
    refuses(name, PLAN, gq.GQ_ERR_SHAPE, n_pages=[0, -1, (1 << 28) + 1], max_pages=[0, 1 << 25], page=[0, 8, 24, 4112],
            n_seq=[0, gq.GQ_MAX_PLAN_SEQ + 1], n_tokens=[-1, (1 << 28) + 1])


def test_embed():
    name = "gq_embed"
    refuses(name, EMBED, gq.GQ_ERR_FORMAT, format=[-1, 4], type=[-1, 3])
    refuses(name, EMBED, gq.GQ_ERR_NULL, W=[None], ids=[None], Y=[None])
    refuses(name, EMBED, gq.GQ_ERR_ALIGN, W=[U], Y=[U], ids=[A + 2], ldy=[257])
    refuses(name, EMBED, gq.GQ_ERR_SHAPE, rows=[0], K=[0, 48, 1 << 25], M=[-1], ldy=[255], scale=[F(NAN), F(INF)])
    assert call(name, EMBED, format=2, K=288, ldy=288) == gq.GQ_ERR_SHAPE   # whole super-blocks
    assert call(name, EMBED, type=1, ldy=260) == gq.GQ_ERR_ALIGN            # 8 bytes off in f16
    assert call(name, EMBED, M=0, ids=None, Y=None) == gq.GQ_OK


@pytest.mark.parametrize("name,good", [("gq_lora_add", LORA), ("gq_lora_add_q8act", LORA8)])
def test_lora(name, good):
    refuses(name, good, gq.GQ_ERR_FORMAT, type=[gq.GQ_TYPE_F32, -1, 3])
    inputs = ("X",) if "X" in good else ("Xq", "dx")
    refuses(name, good, gq.GQ_ERR_NULL, **{p: [None] for p in ("A", "B", "scale", "adapter", "Y0", "Y") + inputs})
    refuses(name, good, gq.GQ_ERR_ALIGN, **{p: [U] for p in ("A", "B", "Y0", "Y", "ws") + inputs}, scale=[A + 2],
            adapter=[A + 2], sequence=[A + 2], ldy0=[34], ldy=[34])
    refuses(name, good, gq.GQ_ERR_SHAPE, n_adapters=[0], rank=[0, 4, 12, 136], rows=[0, 30], K=[0, 48], n_seq=[0], M=[-1],
            ldy0=[28], ldy=[28])
    if "ldx" in good:
        refuses(name, good, gq.GQ_ERR_SHAPE, ldx=[60, -64])
        refuses(name, good, gq.GQ_ERR_ALIGN, ldx=[66])
    assert call(name, good, sequence=None) == gq.GQ_ERR_SHAPE                # five tokens, two requests
    assert call(name, good, Y=good["Y0"], ldy=36) == gq.GQ_ERR_SHAPE         # in place with another stride
    need = gq.gq_lora_workspace_bytes(16, 64, 5)
    assert need > 0
    refuses(name, good, gq.GQ_ERR_WORKSPACE, ws=[None], ws_bytes=[need - 1])
    assert call(name, good, M=0) == gq.GQ_OK


def test_lora_workspace():
    for bad in ((0, 64, 5), (12, 64, 5), (136, 64, 5), (16, 0, 5), (16, 40, 5), (16, 64, 0)):
        assert gq.gq_lora_workspace_bytes(*bad) == 0
    # never more than one sum per 256 elements of a row
    assert gq.gq_lora_workspace_bytes(16, 4096, 1) <= 16 * 16 * 4
    assert gq.gq_lora_workspace_bytes(128, 5376, 1 << 26) >= 128 * 4 << 26   # beyond 32 bits


def test_sample():
    name = "gq_sample"
    refuses(name, SAMPLE, gq.GQ_ERR_FORMAT, type=[-1, 3])
    refuses(name, SAMPLE, gq.GQ_ERR_NULL, logits=[None], u=[None], token=[None])
    refuses(name, SAMPLE, gq.GQ_ERR_ALIGN, **{p: [A + 2] for p in ("t", "k", "p", "m", "u", "token", "prob")}, logits=[A + 2], ws=[U])
    refuses(name, SAMPLE, gq.GQ_ERR_SHAPE, vocab=[0, gq.GQ_MAX_VOCAB + 1], n=[-1, gq.GQ_MAX_SAMPLE_ROWS + 1], ldl=[99])
    need = gq.gq_sample_workspace_bytes(100, 3)
    assert need > 0
    refuses(name, SAMPLE, gq.GQ_ERR_WORKSPACE, ws=[None], ws_bytes=[need - 1])
    assert call(name, SAMPLE, n=0) == gq.GQ_OK
    for bad in ((0, 1), (gq.GQ_MAX_VOCAB + 1, 1), (10, 0), (10, gq.GQ_MAX_SAMPLE_ROWS + 1)):
        assert gq.gq_sample_workspace_bytes(*bad) == 0


def test_the_binding_refuses_what_it_cannot_pass():
    import torch
    x = torch.zeros(3, 128)
    with pytest.raises(ValueError):
        gq.gq_sample(x, 128, 0, None, None, None, None, x, x, None, x, 1, 128, 3)
    with pytest.raises(ValueError):
        gq.gq_embed(1, x, x, 1.0, x, 128, 0, 10, 128, 3)
