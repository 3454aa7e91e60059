"""GPU tests of the paged Q8_0 key/value cache (append, read back) and of the
attention over it, against the plain 64-bit forms of kv_plain.

Tolerances of the attention, per element of o = sum_j w_j v_j with
A = sum_j w_j |v_j| and Z = the row's largest scale * sum |q k_j|:
  A score that is off by delta changes every weight by at most a factor
  e^(+-2 delta), and with it o by at most 2.1 delta A (delta small).
  f32: operands of 22 bits and f32 sums: delta <= 2^-20 Z (two operands of
  2^-22 each, the sum of up to 256 products in f32 and its scaling); the
  probabilities, their products with the scales and the sums of at most 2^7
  tensor-core additions of 2^-23 each: 2^-16 A.
  16 bits: operands rounded to 11 bits (2^-12 each): delta <= 2^-10 Z for q k
  and 2^-10 A for p v, and the result's own rounding.
The 2-norm of the error over the whole output, where roundings average, is
held to 1e-5 of the output's for f32 as the interface promises, and to the
unit roundoff of the type for the others."""

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import kv_plain as kp
from gpu_util import dev, torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": gq.GQ_TYPE_F32, "f16": gq.GQ_TYPE_F16, "bf16": gq.GQ_TYPE_BF16}
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def tt(typ):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[typ]


def lists(batch):
    return dev(batch.table), dev(np.asarray(batch.kv_len, np.int32)), dev(batch.starts)


def sizes(batch):
    return (batch.cache.shape[0], batch.table.shape[1], batch.page, batch.kv_heads, batch.dim, len(batch.kv_len),
            batch.n_tokens)


def token_array(x, typ, pad=0):
    """[tokens][heads][dim] f32 -> (device rows with `pad` extra elements between rows, the values that they hold)."""
    t = torch()
    n = x.shape[0]
    full = t.full((n, x[0].size + pad if n else pad), float("nan"), dtype=tt(typ), device="cuda")
    view = full[:, :x[0].size] if n else full
    if n:
        view.copy_(dev(x.reshape(n, -1)).to(tt(typ)))
    return view, view.float().cpu().numpy().reshape(x.shape)


def random_batch(kv_len, counts, kv_heads, dim, page, rng, fill=0, v_scale=None):
    """A batch whose cached tokens are all written."""
    batch = kp.make(kv_len, counts, kv_heads, dim, page, rng, fill=fill)
    for b, kv in enumerate(kv_len):
        for p in range(kv):
            k = rng.standard_normal((kv_heads, dim)).astype(np.float32)
            v = rng.standard_normal((kv_heads, dim)).astype(np.float32)
            if v_scale is not None:
                v = v * np.float32(v_scale(p))
            kp.write(batch, b, p, k, v)
    return batch


# ---------------------------------------------------------------- append

APPEND = [
    # kv_len, new tokens, kv heads, dim, page
    ([1], [1], 1, 64, 16),
    ([37, 5, 0, 64], [3, 5, 0, 1], 2, 128, 16),
    ([130, 33], [130, 17], 8, 128, 64),
    ([19, 16, 15, 32, 47], [18, 1, 2, 16, 30], 4, 256, 32),
    ([700], [523], 2, 64, 128),
    ([3 + b for b in range(40)], [1 + b % 3 for b in range(40)], 1, 128, 16),
]


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_writes_the_new_tokens_and_nothing_else(case, typ):
    kv_len, counts, hk, dim, page = APPEND[case]
    rng = np.random.default_rng(900 + case)
    batch = kp.make(kv_len, counts, hk, dim, page, rng, fill=0xA5)
    k = rng.standard_normal((batch.n_tokens, hk, dim)).astype(np.float32)
    v = (rng.standard_normal((batch.n_tokens, hk, dim)) * 10.0 ** rng.integers(-6, 5, (batch.n_tokens, hk, 1))).astype(np.float32)
    kd, k = token_array(k, typ, pad=8)
    vd, v = token_array(v, typ, pad=24)
    cache = dev(batch.cache)
    gq.gq_kv_append_q8_0(kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], cache, *lists(batch), *sizes(batch))
    for b in range(len(kv_len)):
        for i, p in enumerate(batch.positions(b)):
            kp.write(batch, b, p, k[batch.starts[b] + i], v[batch.starts[b] + i])
    assert np.array_equal(cache.cpu().numpy(), batch.cache)
    assert gq.gq_device_status() == gq.GQ_OK


def test_append_large_call_matches_small_ones():
    """The four-units-a-warp form (large calls) against single-token calls."""
    t = torch()
    rng = np.random.default_rng(917)
    hk, dim, page, n = 8, 128, 64, 1531
    batch = kp.make([n + 7], [n], hk, dim, page, rng)
    k = dev(rng.standard_normal((n, hk * dim)).astype(np.float32))
    v = dev(rng.standard_normal((n, hk * dim)).astype(np.float32))
    one, many = dev(batch.cache), dev(batch.cache)
    gq.gq_kv_append_q8_0(k, k.stride(0), v, v.stride(0), gq.GQ_TYPE_F32, one, *lists(batch), *sizes(batch))
    table = dev(batch.table)
    start = dev(np.array([0, 1], np.int32))
    for i in range(n):
        gq.gq_kv_append_q8_0(k[i:i + 1], k.stride(0), v[i:i + 1], v.stride(0), gq.GQ_TYPE_F32, many, table,
                             t.tensor([8 + i], dtype=t.int32, device="cuda"), start, *sizes(batch)[:5], 1, 1)
    assert t.equal(one, many)


def test_append_extreme_values():
    """Saturation at fp16's range, underflow of the scale, infinities, NaN, negative zero."""
    dim = 64
    rng = np.random.default_rng(921)
    rows = [np.full(dim, 3e38), np.full(dim, -65504.0), np.full(dim, 1e-9), np.zeros(dim), np.full(dim, -0.0),
            np.where(np.arange(dim) % 7 == 0, np.inf, 1.0), np.where(np.arange(dim) % 9 == 0, -np.inf, -2.0),
            np.where(np.arange(dim) % 5 == 0, np.nan, rng.standard_normal(dim)), np.full(dim, np.nan),
            rng.standard_normal(dim) * 127 * 2.0 ** -24, np.arange(dim) - 31.5, 127 * 515.5 * np.sign(rng.standard_normal(dim))]
    x = np.stack(rows).astype(np.float32)[:, None, :]
    n = len(rows)
    batch = kp.make([n], [n], 1, dim, 16, rng)
    k, _ = token_array(x, "f32")
    v, _ = token_array(x[::-1].copy(), "f32")
    cache = dev(batch.cache)
    gq.gq_kv_append_q8_0(k, k.stride(0), v, v.stride(0), gq.GQ_TYPE_F32, cache, *lists(batch), *sizes(batch))
    for p in range(n):
        kp.write(batch, 0, p, x[p], x[n - 1 - p])
    assert np.array_equal(cache.cpu().numpy(), batch.cache)


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_read_gives_the_cached_values(case, typ):
    t = torch()
    kv_len, counts, hk, dim, page = APPEND[case]
    rng = np.random.default_rng(930 + case)
    batch = random_batch(kv_len, counts, hk, dim, page, rng, fill=0xFF)
    n, w = batch.n_tokens, hk * dim
    full = [t.full((n + 2, w + 8), 7.5, dtype=tt(typ), device="cuda") for _ in range(2)]
    k, v = (f[1:n + 1, :w] for f in full)
    gq.gq_kv_read_q8_0(dev(batch.cache), *lists(batch), k, k.stride(0), v, v.stride(0), TYPES[typ], *sizes(batch))
    kr, vr = (np.concatenate(x) for x in zip(*(kp.values(batch, b, batch.positions(b)) for b in range(len(kv_len)))))
    for got, ref, f in ((k, kr, full[0]), (v, vr, full[1])):
        want = t.from_numpy(ref.reshape(n, w)).float().to(tt(typ))  # exact in f32, rounded once
        assert t.equal(got.cpu(), want)
        assert bool((f[0] == 7.5).all()) and bool((f[-1] == 7.5).all()) and bool((f[:, w:] == 7.5).all())
    assert gq.gq_device_status() == gq.GQ_OK


# ---------------------------------------------------------------- attention

def check_attention(batch, heads, typ, rng, window=0, softcap=0.0, pad=0, q_scale=1.5, scale=None, q=None, ws=None,
                    norm=True):
    t = torch()
    dim, n = batch.dim, batch.n_tokens
    scale = dim ** -0.5 if scale is None else scale
    if q is None:
        q = (rng.standard_normal((n, heads, dim)) * q_scale).astype(np.float32)
    qd, q = token_array(q, typ, pad=pad)
    full = t.full((n + 2, heads * dim + pad), 7.5, dtype=tt(typ), device="cuda")
    out = full[1:n + 1, :heads * dim]
    if ws is None:
        ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, batch.kv_heads, dim), dtype=t.uint8, device="cuda")
    gq.gq_kv_attention_q8_0(qd, qd.stride(0), dev(batch.cache), *lists(batch), out, out.stride(0), TYPES[typ], scale,
                            softcap, window, ws, ws.numel(), heads, *sizes(batch))
    got = out.float().cpu().numpy().astype(np.float64).reshape(n, heads, dim)
    f = full.float().cpu().numpy()
    assert (f[0] == 7.5).all() and (f[-1] == 7.5).all() and (f[:, heads * dim:] == 7.5).all(), "written outside the rows"
    ref, a, mag = kp.attention(batch, q, scale, softcap, window)
    z = mag[..., None]
    if typ == "f32":
        bound = (2.1 * 2.0 ** -20 * z + 2.0 ** -16) * a
    else:
        bound = (2.1 * 2.0 ** -10 * z + 2.0 ** -10) * a + ROUND[typ] * np.abs(ref) + 2.0 ** -24
    err = np.abs(got - ref)
    assert np.all(err <= bound), (float((err / np.maximum(bound, 1e-300)).max()), np.argwhere(~(err <= bound))[:4])
    if norm and np.linalg.norm(ref) > 0:
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= (1e-5 if typ == "f32" else ROUND[typ]), rel
    return out


ATTENTION = [
    # kv_len, new tokens, heads, kv heads, dim, page, window, softcap
    ([1], [1], 1, 1, 64, 16, 0, 0.0),                                        # one token sees itself
    ([129], [1], 8, 1, 128, 16, 0, 0.0),
    ([33, 1, 0, 250, 16, 17], [1, 1, 0, 1, 1, 1], 8, 2, 128, 32, 0, 0.0),    # a sequence without tokens
    ([70, 16, 3], [5, 16, 3], 6, 2, 64, 16, 0, 0.0),                         # groups of three, whole prompts
    ([300, 90], [7, 90], 7, 1, 256, 64, 0, 30.0),
    ([260, 41], [4, 41], 4, 4, 128, 16, 13, 0.0),                            # one head a group, a window inside a record
    ([513, 64], [33, 64], 16, 2, 128, 64, 100, 50.0),
    ([400], [150], 10, 2, 64, 128, 0, 0.0),
    ([150], [150], 4, 1, 256, 16, 1, 0.0),                                   # a window of the token itself
    ([2, 40], [5, 40], 4, 2, 128, 16, 0, 0.0),                               # three rows before position 0: nothing to read
    ([1500, 1100], [1, 1], 16, 1, 128, 64, 0, 0.0),                          # sixteen heads a group
    ([600, 300], [70, 300], 32, 4, 128, 64, 0, 0.0),                         # larger chunks
    ([517], [261], 8, 8, 256, 32, 200, 0.0),
    ([700], [333], 5, 1, 64, 16, 0, 20.0),
]


@pytest.mark.parametrize("typ", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(case, typ):
    kv_len, counts, heads, hk, dim, page, window, cap = ATTENTION[case]
    rng = np.random.default_rng(950 + case)
    # whatever lies in the pages beyond the cached tokens (NaN scales) must not matter
    batch = random_batch(kv_len, counts, hk, dim, page, rng, fill=0xFF)
    check_attention(batch, heads, typ, rng, window, cap, pad=8 * (case % 3))
    assert gq.gq_device_status() == gq.GQ_OK


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[1], [90]])
def test_attention_values_of_very_different_size(counts, typ):
    """Value scales over fp16's whole range: the largest tokens must not push the others out of range."""
    rng = np.random.default_rng(970)
    batch = random_batch([200], counts, 1, 128, 16, rng, v_scale=lambda p: 10.0 ** ((p * 7) % 11 - 6))
    check_attention(batch, 4, typ, rng)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("size", [1e-12, 1e12])
def test_attention_queries_of_any_size(size, n, typ):
    """Queries far outside fp16's range, with a scale that brings the scores back."""
    rng = np.random.default_rng(971)
    batch = random_batch([120], [n], 2, 64, 16, rng)
    check_attention(batch, 4, typ, rng, q_scale=size, scale=float(0.125 / size))


@pytest.mark.parametrize("n", [1, 80])
def test_attention_one_strong_key_and_many_weak_ones(n):
    """Probabilities far below fp16's smallest number still count together."""
    rng = np.random.default_rng(972)
    batch = random_batch([1400], [n], 1, 64, 64, rng)
    strong = np.zeros((1, 64), np.float32)
    strong[0, :] = 3.0
    kp.write(batch, 0, 700, strong, np.full((1, 64), 0.01, np.float32))
    q = np.full((n, 2, 64), 0.5, np.float32) + (rng.standard_normal((n, 2, 64)) * 0.02).astype(np.float32)
    check_attention(batch, 2, "f32", rng, q=q)


@pytest.mark.parametrize("n", [1, 3, 100])
def test_attention_a_nonfinite_query_stays_in_its_row(n):
    t = torch()
    rng = np.random.default_rng(973)
    batch = random_batch([150], [n], 2, 128, 16, rng)
    heads = 4
    q = rng.standard_normal((n, heads, 128)).astype(np.float32)
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, 2, 128), dtype=t.uint8, device="cuda")
    cache = dev(batch.cache)

    def run(x):
        out = t.empty((n, heads * 128), device="cuda")
        xd = dev(x.reshape(n, -1))
        gq.gq_kv_attention_q8_0(xd, xd.stride(0), cache, *lists(batch), out, out.stride(0), gq.GQ_TYPE_F32, 0.1, 0.0, 0,
                                ws, ws.numel(), heads, *sizes(batch))
        return out.cpu().numpy().reshape(n, heads, 128)

    clean = run(q)
    for bad in (np.nan, np.inf):
        p = q.copy()
        p[n // 2, 1, 17] = bad
        got = run(p)
        assert np.isnan(got[n // 2, 1]).all()
        got[n // 2, 1] = clean[n // 2, 1]
        assert np.array_equal(got, clean)


@pytest.mark.parametrize("typ,counts", [("bf16", [1, 1, 1]), ("f32", [1, 1, 1]), ("bf16", [200, 17, 3]), ("f32", [200, 17, 3])])
def test_attention_is_deterministic_and_leaves_the_workspace_ready(typ, counts):
    t = torch()
    rng = np.random.default_rng(974)
    batch = random_batch([900, 333, 40], counts, 2, 128, 16, rng)
    heads = 8
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, 2, 128), dtype=t.uint8, device="cuda")
    q = rng.standard_normal((batch.n_tokens, heads, 128)).astype(np.float32)
    first = check_attention(batch, heads, typ, rng, q=q, ws=ws)
    other = random_batch([77], [5], 2, 128, 16, rng)
    check_attention(other, heads, typ, rng, ws=ws)  # another problem through the same workspace
    for _ in range(3):
        assert t.equal(check_attention(batch, heads, typ, rng, q=q, ws=ws), first)


@pytest.mark.parametrize("n", [1, 64])
def test_attention_on_another_stream_and_in_a_graph(n):
    """The lists are read on the device: a captured call follows lengths that change after the capture."""
    t = torch()
    rng = np.random.default_rng(975)
    kv = 180
    batch = random_batch([kv], [n], 2, 128, 16, rng)
    heads = 8
    q = dev(rng.standard_normal((n, heads * 128)).astype(np.float32))
    out = t.zeros((n, heads * 128), device="cuda")
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, 2, 128), dtype=t.uint8, device="cuda")
    cache = dev(batch.cache)
    table, kv_len, start = lists(batch)
    args = (q, q.stride(0), cache, table, kv_len, start, out, out.stride(0), gq.GQ_TYPE_F32, 0.1, 0.0, 0, ws, ws.numel(),
            heads, *sizes(batch))
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        gq.gq_kv_attention_q8_0(*args)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        gq.gq_kv_attention_q8_0(*args)
    for length in (kv, n + 3, kv - 50):
        kv_len.fill_(length)
        graph.replay()
        t.cuda.synchronize()
        batch.kv_len = [length]
        ref, a, mag = kp.attention(batch, q.cpu().numpy().reshape(n, heads, 128), 0.1)
        err = np.abs(out.cpu().numpy().reshape(ref.shape) - ref)
        assert np.all(err <= (2.1 * 2.0 ** -20 * mag[..., None] + 2.0 ** -16) * a)


@pytest.mark.parametrize("n", [1, 70])
def test_pages_and_lengths_out_of_range_are_reported_and_not_followed(n):
    t = torch()
    rng = np.random.default_rng(976)
    batch = random_batch([100, 50], [n, 1], 2, 64, 16, rng)
    heads = 4
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, 2, 64), dtype=t.uint8, device="cuda")
    q = dev(rng.standard_normal((n + 1, heads * 64)).astype(np.float32))
    cache = dev(batch.cache)
    out = t.empty((n + 1, heads * 64), device="cuda")
    table, kv_len, start = lists(batch)

    def call(table, kv_len):
        gq.gq_kv_attention_q8_0(q, q.stride(0), cache, table, kv_len, start, out, out.stride(0), gq.GQ_TYPE_F32, 0.1, 0.0,
                                0, ws, ws.numel(), heads, *sizes(batch))
        return out.cpu().clone()

    good = call(table, kv_len)
    assert gq.gq_device_status() == gq.GQ_OK
    for wrong in (-1, batch.cache.shape[0], 2 ** 31 - 1):
        bad = table.clone()
        bad[0, 2] = wrong
        got = call(bad, kv_len)
        assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
        assert t.equal(got[n:], good[n:]) and bool(t.isfinite(got).all())
        # the page's tokens are left out
        other = kp.Batch([84], [n], 2, 64, 16, np.delete(batch.table[:1], 2, axis=1), batch.cache)
        ref, a, mag = kp.attention(other, q[:n].cpu().numpy().reshape(n, heads, 64), 0.1)
        rows = [i for i in range(n) if 100 - n + i >= 48]  # queries past the page see the same tokens as without it
        err = np.abs(got[:n].numpy().reshape(ref.shape) - ref)[rows]
        assert np.all(err <= ((2.1 * 2.0 ** -20 * mag[..., None] + 2.0 ** -16) * a)[rows])
        k = t.full((n + 1, 128), 7.5, device="cuda")
        v = t.full((n + 1, 128), 7.5, device="cuda")
        long = t.tensor([0, n, n + 1], dtype=t.int32, device="cuda")
        gq.gq_kv_read_q8_0(cache, bad, kv_len, long, k, 128, v, 128, gq.GQ_TYPE_F32, *sizes(batch))
        hit = [i for i in range(n) if (100 - n + i) // 16 == 2]
        assert bool((k[hit] == 0).all()) and bool((v[hit] == 0).all())
        assert gq.gq_device_status() == (gq.GQ_ERR_SHAPE if hit else gq.GQ_OK)
        before = cache.clone()
        gq.gq_kv_append_q8_0(k, 128, v, 128, gq.GQ_TYPE_F32, before, bad, kv_len, long, *sizes(batch))
        assert gq.gq_device_status() == (gq.GQ_ERR_SHAPE if hit else gq.GQ_OK)
    kv_len[0] = 10 ** 6
    got = call(table, kv_len)
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    # the other sequence's keys may be split at other places now
    assert t.allclose(got[n:], good[n:], rtol=0, atol=1e-5)


def test_append_then_attend_agrees_with_attention_over_the_written_values():
    """The path of a decode step: append a token, attend, step by step and as one chunk."""
    t = torch()
    rng = np.random.default_rng(977)
    hk, heads, dim, page, total = 2, 8, 128, 16, 45
    batch = kp.make([total], [total], hk, dim, page, rng, fill=0xFF)
    x = dev(rng.standard_normal((total, (heads + 2 * hk) * dim)).astype(np.float32))  # one projection's rows
    q, k, v = x[:, :heads * dim], x[:, heads * dim:(heads + hk) * dim], x[:, (heads + hk) * dim:]
    table = dev(batch.table)
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, hk, dim), dtype=t.uint8, device="cuda")

    def step(cache, r0, r1, out):
        kv = t.tensor([r1], dtype=t.int32, device="cuda")
        st = t.tensor([0, r1 - r0], dtype=t.int32, device="cuda")
        n = (*sizes(batch)[:5], 1, r1 - r0)
        gq.gq_kv_append_q8_0(k[r0:r1], k.stride(0), v[r0:r1], v.stride(0), gq.GQ_TYPE_F32, cache, table, kv, st, *n)
        gq.gq_kv_attention_q8_0(q[r0:r1], q.stride(0), cache, table, kv, st, out[r0:r1], out.stride(0), gq.GQ_TYPE_F32,
                                dim ** -0.5, 0.0, 0, ws, ws.numel(), heads, *n)

    whole, steps = (t.empty((total, heads * dim), device="cuda") for _ in range(2))
    c1, c2 = dev(batch.cache), dev(batch.cache)
    step(c1, 0, total, whole)
    for i in range(total):
        step(c2, i, i + 1, steps)
    assert t.equal(c1, c2)
    batch.cache = c1.cpu().numpy()
    ref, a, mag = kp.attention(batch, q.cpu().numpy().reshape(total, heads, dim), dim ** -0.5)
    bound = (2.1 * 2.0 ** -20 * mag[..., None] + 2.0 ** -16) * a
    for got in (whole, steps):
        assert np.all(np.abs(got.cpu().numpy().reshape(ref.shape) - ref) <= bound)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_many_sequences(typ):
    """More sequences than a search step, a plan's threads or its warps look at in one go."""
    t = torch()
    rng = np.random.default_rng(980)
    n_seq = 1100
    kv_len = [int(x) for x in rng.integers(1, 40, n_seq)]
    counts = [int(rng.integers(0, 3)) if kv > 2 else kv for kv in kv_len]
    batch = kp.make(kv_len, [kv for kv in kv_len], 1, 64, 16, rng)
    k = rng.standard_normal((batch.n_tokens, 1, 64)).astype(np.float32)
    v = rng.standard_normal((batch.n_tokens, 1, 64)).astype(np.float32)
    kd, k = token_array(k, typ)
    vd, v = token_array(v, typ)
    cache = dev(batch.cache)
    gq.gq_kv_append_q8_0(kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], cache, *lists(batch), *sizes(batch))
    for b in range(n_seq):
        for i, p in enumerate(batch.positions(b)):
            kp.write(batch, b, p, k[batch.starts[b] + i], v[batch.starts[b] + i])
    assert np.array_equal(cache.cpu().numpy(), batch.cache)
    gq.gq_kv_read_q8_0(cache, *lists(batch), kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], *sizes(batch))
    ref = np.concatenate([kp.values(batch, b, batch.positions(b))[0] for b in range(n_seq)]).reshape(-1, 64)
    assert t.equal(kd.cpu(), t.from_numpy(ref).float().to(tt(typ)))
    batch.counts = counts
    check_attention(batch, 2, typ, rng)
    # and in the form for many rows: 30 sequences of 70 to 90 rows
    chunk = random_batch([int(x) for x in rng.integers(90, 200, 30)], [int(x) for x in rng.integers(70, 90, 30)], 1, 64, 16, rng)
    check_attention(chunk, 1, typ, rng)
    assert gq.gq_device_status() == gq.GQ_OK


@pytest.mark.parametrize("typ,dim", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f16", 64), ("f32", 64), ("f32", 128)])
def test_chunk_results_do_not_vary(typ, dim):
    """The same call many times over gives the same bits: a stage refilled too early, or a wait for the wrong
    phase, would show as now and then another row."""
    t = torch()
    rng = np.random.default_rng(981)
    batch = random_batch([700, 390, 1100], [300, 390, 90], 2, dim, 16, rng)
    heads = 4
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, 2, dim), dtype=t.uint8, device="cuda")
    q = (rng.standard_normal((batch.n_tokens, heads, dim)) * 1.5).astype(np.float32)
    first = check_attention(batch, heads, typ, rng, q=q, ws=ws)
    qd, _ = token_array(q, typ)
    out = t.empty((batch.n_tokens, heads * dim), dtype=tt(typ), device="cuda")
    cache, ls = dev(batch.cache), lists(batch)
    for _ in range(200):
        out.fill_(float("nan"))
        gq.gq_kv_attention_q8_0(qd, qd.stride(0), cache, *ls, out, out.stride(0), TYPES[typ], dim ** -0.5, 0.0, 0, ws, ws.numel(),
                                heads, *sizes(batch))
        assert t.equal(out, first)


@pytest.mark.parametrize("n", [1, 70])
def test_a_cache_beyond_32_bit_offsets(n):
    """Pages more than 2^32 bytes into the cache, against the same pages at its start."""
    t = torch()
    rng = np.random.default_rng(982)
    batch = random_batch([150], [n], 1, 64, 16, rng)
    heads, page_bytes = 2, 34 * 64
    small = dev(batch.cache)
    n_small = batch.cache.shape[0]
    n_large = 2 ** 32 // page_bytes + 1000
    large = t.empty(n_large * page_bytes, dtype=t.uint8, device="cuda")
    shift = n_large - n_small
    large[shift * page_bytes:].copy_(small.reshape(-1))
    table, kv_len, start = lists(batch)
    far = t.where(table >= 0, table + shift, table).to(t.int32)
    x = dev(rng.standard_normal((n, 64)).astype(np.float32))
    q = dev(rng.standard_normal((n, heads * 64)).astype(np.float32))
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(heads, 1, 64), dtype=t.uint8, device="cuda")
    got = []
    for cache, tab, pages in ((small, table, n_small), (large, far, n_large)):
        s = (pages, *sizes(batch)[1:])
        gq.gq_kv_append_q8_0(x, 64, x, 64, gq.GQ_TYPE_F32, cache, tab, kv_len, start, *s)
        k, v = t.empty_like(x), t.empty_like(x)
        gq.gq_kv_read_q8_0(cache, tab, kv_len, start, k, 64, v, 64, gq.GQ_TYPE_F32, *s)
        outs = [k, v]
        for typ in ("f32", "bf16"):
            qt = q.to(tt(typ))
            o = t.empty_like(qt)
            gq.gq_kv_attention_q8_0(qt, qt.stride(0), cache, tab, kv_len, start, o, o.stride(0), TYPES[typ], 0.125, 0.0, 0, ws,
                                    ws.numel(), heads, *s)
            outs.append(o)
        got.append(outs)
    assert all(t.equal(a, b) for a, b in zip(*got))
    assert t.equal(large[shift * page_bytes:], small.reshape(-1))
    assert gq.gq_device_status() == gq.GQ_OK


@pytest.mark.parametrize("n", [2, 70])
def test_rows_beyond_the_token_arrays_are_reported_and_not_touched(n):
    t = torch()
    rng = np.random.default_rng(983)
    batch = random_batch([100, 90], [n, n], 1, 64, 16, rng)
    cache = dev(batch.cache)
    table, kv_len, start = lists(batch)
    start[2] += 5  # five rows more than the arrays have
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(1, 1, 64), dtype=t.uint8, device="cuda")
    full = t.full((2 * n + 8, 64), 7.5, device="cuda")
    x = full[:2 * n]
    gq.gq_kv_read_q8_0(cache, table, kv_len, start, x, 64, x, 64, gq.GQ_TYPE_F32, *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    q = dev(rng.standard_normal((2 * n, 64)).astype(np.float32))
    gq.gq_kv_attention_q8_0(q, 64, cache, table, kv_len, start, x, 64, gq.GQ_TYPE_F32, 0.1, 0.0, 0, ws, ws.numel(), 1, *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    gq.gq_kv_append_q8_0(q, 64, q, 64, gq.GQ_TYPE_F32, cache, table, kv_len, start, *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    assert bool((full[2 * n:] == 7.5).all())


def test_calls_without_tokens_do_nothing():
    t = torch()
    rng = np.random.default_rng(978)
    batch = random_batch([20], [0], 1, 64, 16, rng)
    cache = dev(batch.cache)
    x = t.full((1, 64), 7.5, device="cuda")
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(1, 1, 64), dtype=t.uint8, device="cuda")
    gq.gq_kv_append_q8_0(x, 64, x, 64, gq.GQ_TYPE_F32, cache, *lists(batch), *sizes(batch))
    gq.gq_kv_read_q8_0(cache, *lists(batch), x, 64, x, 64, gq.GQ_TYPE_F32, *sizes(batch))
    gq.gq_kv_attention_q8_0(x, 64, cache, *lists(batch), x, 64, gq.GQ_TYPE_F32, 1.0, 0.0, 0, ws, ws.numel(), 1, *sizes(batch))
    assert np.array_equal(cache.cpu().numpy(), batch.cache) and bool((x == 7.5).all())
