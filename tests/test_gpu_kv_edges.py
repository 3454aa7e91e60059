"""GPU tests of the paged Q8_0 cache and its attention at the edges of what
the interface allows: lists that lead outside the cache or the token arrays,
windows beyond every position, strong keys with small values, scores of any
size, calls without tokens, scales next to a tie of the fp16 rounding.

The reference is written here for single rows, in 64 bits, on kv_plain's
cache; tolerances as derived in test_gpu_kv, with what is said at each test."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import kv_plain as kp
from gpu_util import dev, torch
from test_gpu_kv import ROUND, TYPES, check_attention, lists, random_batch, sizes, token_array, tt

pytestmark = pytest.mark.gpu


def row_attention(batch, b, q, lo, hi, scale, softcap=0.0):
    """One query row [heads][dim] over the positions lo .. hi - 1 of sequence b: (o, sum w |v|), zeros where there is none."""
    heads = q.shape[0]
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    if hi <= lo:
        return o, a
    k, v = kp.values(batch, b, range(lo, hi))
    for h in range(heads):
        g = h // (heads // batch.kv_heads)
        s = scale * (k[:, g] @ q[h].astype(np.float64))
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        w = np.exp(s - s.max())
        w /= w.sum()
        o[h], a[h] = w @ v[:, g], w @ np.abs(v[:, g])
    return o, a


def attend(batch, qd, typ, heads, scale, window=0, softcap=0.0, ls=None, out=None):
    t = torch()
    out = t.full((qd.shape[0], heads * batch.dim), 7.5, dtype=tt(typ), device="cuda") if out is None else out
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, batch.kv_heads, batch.dim), dtype=t.uint8, device="cuda")
    gq.gq_kv_attention_q8_0(qd, qd.stride(0), dev(batch.cache), *(ls or lists(batch)), out, out.stride(0), TYPES[typ], scale,
                            softcap, window, ws, ws.numel(), heads, *sizes(batch))
    return out.float().cpu().numpy().astype(np.float64).reshape(qd.shape[0], heads, batch.dim)


# ---------------------------------------------------------------- windows

@pytest.mark.parametrize("typ,dim", [("f32", 64), ("f32", 256), ("bf16", 128), ("bf16", 256)])
@pytest.mark.parametrize("counts", [[5, 1], [90, 90]])
def test_a_window_beyond_every_position_hides_nothing(counts, typ, dim):
    """Rows before position 0 (kv_len below the new tokens' number) included: their windows begin far below 0."""
    rng = np.random.default_rng(1000)
    batch = random_batch([2, 90], counts, 1, dim, 16, rng, fill=0xFF)
    q, _ = token_array((rng.standard_normal((batch.n_tokens, 2, dim))).astype(np.float32), typ)
    want = attend(batch, q, typ, 2, 0.1)
    for window in (2 ** 31 - 1, 2 ** 31 - 60, 2 ** 30, 2 ** 28):
        assert np.array_equal(attend(batch, q, typ, 2, 0.1, window=window), want), window
    check_attention(batch, 2, typ, rng, window=2 ** 31 - 1)
    assert gq.gq_device_status() == gq.GQ_OK
