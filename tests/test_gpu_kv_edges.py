"""GPU tests of the paged Q8_0 cache and its attention at the edges of what
the interface allows: lists that lead outside the cache or the token arrays,
windows beyond every position, strong keys with small values, scores of any
size, calls without tokens, scales next to a tie of the fp16 rounding.

The reference is written here for single rows, in 64 bits, on kv_plain's
cache; tolerances as derived in test_gpu_kv, with what is said at each test."""

import functools

import numpy as np
import pytest

import block_quantized_matvec_gq_gb300 as gq
import kv_plain as kp
from gpu_util import dev, torch
from test_gpu_kv import ROUND, TYPES, check_attention, lists, random_batch, sizes, token_array, tt

pytestmark = pytest.mark.gpu


_values = {}


def row_attention(batch, b, q, lo, hi, scale, softcap=0.0):
    """One query row [heads][dim] over the positions lo .. hi - 1 of sequence b: (o, sum w |v|), zeros where there is none."""
    heads = q.shape[0]
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    if hi <= lo:
        return o, a
    key = (id(batch), b)
    if _values.get("of") != key:  # the last sequence's cached values, for the rows that follow
        _values.update(of=key, batch=batch, kv=kp.values(batch, b, range(min(batch.kv_len[b], batch.table.shape[1] * batch.page))))
    k, v = (x[lo:hi] for x in _values["kv"])
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


# ---------------------------------------------------------------- lists that lead outside

def full_batch(kv_len, counts, kv_heads, dim, page, rng):
    """A batch whose table has no entry to spare: the first sequence fills it."""
    batch = random_batch(kv_len, counts, kv_heads, dim, page, rng)
    batch.table = np.ascontiguousarray(batch.table[:, :-1])
    assert batch.table.shape[1] * page == kv_len[0]
    return batch


# kv_len past the table's last position, new tokens of that sequence, window
LONG = [(1, 1, 0), (1, 3, 0), (3, 3, 20), (7, 5, 0), (2, 90, 0), (100, 90, 40), (10 ** 6, 70, 0), (2 ** 31 - 1 - 96, 2, 0),
        (40, 1, 5), (17, 9, 16)]


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("over,n,window", LONG)
def test_a_length_past_the_table_moves_no_token(over, n, window, typ):
    """kv_len beyond max_pages * page_tokens: rows keep their positions, those past the last one are not written, read
    as zeros and not attended to, and nothing that was cached changes."""
    t = torch()
    rng = np.random.default_rng(1010)
    hk, heads, dim, page, room = 2, 4, 64, 16, 96
    batch = full_batch([room, 40], [n, 3], hk, dim, page, rng)
    table, kv_len, start = lists(batch)
    kv_len[0] = room + over
    ls = (table, kv_len, start)
    pos = [room + over - n + i for i in range(n)] + [37, 38, 39]
    seq = [0] * n + [1] * 3
    k = rng.standard_normal((n + 3, hk, dim)).astype(np.float32)
    v = rng.standard_normal((n + 3, hk, dim)).astype(np.float32)
    kd, k = token_array(k, typ)
    vd, v = token_array(v, typ)
    cache = dev(batch.cache)
    gq.gq_kv_append_q8_0(kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], cache, *ls, *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    for i, (b, p) in enumerate(zip(seq, pos)):
        if 0 <= p < room:
            kp.write(batch, b, p, k[i], v[i])
    assert np.array_equal(cache.cpu().numpy(), batch.cache)

    kd.fill_(7.5), vd.fill_(7.5)
    gq.gq_kv_read_q8_0(cache, *ls, kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    for i, (b, p) in enumerate(zip(seq, pos)):
        want = kp.values(batch, b, [p]) if p < room else np.zeros((2, 1, hk, dim))
        for got, ref in zip((kd, vd), want):
            assert t.equal(got[i].cpu(), t.from_numpy(ref.reshape(-1)).float().to(tt(typ))), (i, p)

    q, qh = token_array((rng.standard_normal((n + 3, heads, dim)) * 1.5).astype(np.float32), typ)
    got = attend(batch, q, typ, heads, 0.125, window=window, ls=ls)
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    for i, (b, p) in enumerate(zip(seq, pos)):
        lo = max(0, p - window + 1) if window else 0
        ref, a = row_attention(batch, b, qh[i], lo, min(p + 1, room), 0.125)
        # scores up to 8 sqrt(64) * 0.125 * 1.5 in size: Z < 32
        bound = (2.1 * 2.0 ** -15 + 2.0 ** -16) * a if typ == "f32" else (2.1 * 2.0 ** -5 + 2.0 ** -10) * a + ROUND[typ] * np.abs(ref)
        assert np.all(np.abs(got[i] - ref) <= bound), (i, p)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("n,extra,window", [(2, 5, 0), (3, 1, 0), (70, 5, 0), (70, 33, 11), (90, 2 ** 31 - 200, 0)])
def test_rows_past_the_token_arrays_move_no_token(n, extra, window, typ):
    """A q_start beyond n_tokens: the rows that the arrays have keep the positions that the lists give them."""
    t = torch()
    rng = np.random.default_rng(1011)
    hk, heads, dim, page = 1, 2, 64, 16
    batch = random_batch([100, 96], [n, n], hk, dim, page, rng)
    table, kv_len, start = lists(batch)
    start[2] += extra
    ls = (table, kv_len, start)
    pos = [100 - n + i for i in range(n)] + [96 - (n + extra) + i for i in range(n)]
    seq = [0] * n + [1] * n
    k = rng.standard_normal((2 * n, hk, dim)).astype(np.float32)
    kd, k = token_array(k, typ)
    vd = -kd
    cache = dev(batch.cache)
    gq.gq_kv_append_q8_0(kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], cache, *ls, *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    for i, (b, p) in enumerate(zip(seq, pos)):
        if p >= 0:
            kp.write(batch, b, p, k[i], -k[i])
    assert np.array_equal(cache.cpu().numpy(), batch.cache)
    kd.fill_(7.5), vd.fill_(7.5)
    gq.gq_kv_read_q8_0(cache, *ls, kd, kd.stride(0), vd, vd.stride(0), TYPES[typ], *sizes(batch))
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    for i, (b, p) in enumerate(zip(seq, pos)):
        want = kp.values(batch, b, [p]) if p >= 0 else np.zeros((2, 1, hk, dim))
        for got, ref in zip((kd, vd), want):
            assert t.equal(got[i].cpu(), t.from_numpy(ref.reshape(-1)).float().to(tt(typ))), (i, p)
    q, qh = token_array((rng.standard_normal((2 * n, heads, dim)) * 1.5).astype(np.float32), typ)
    got = attend(batch, q, typ, heads, 0.125, window=window, ls=ls)
    assert gq.gq_device_status() == gq.GQ_ERR_SHAPE
    for i, (b, p) in enumerate(zip(seq, pos)):
        lo = max(0, p - window + 1) if window else 0
        ref, a = row_attention(batch, b, qh[i], lo, p + 1, 0.125)
        bound = (2.1 * 2.0 ** -15 + 2.0 ** -16) * a if typ == "f32" else (2.1 * 2.0 ** -5 + 2.0 ** -10) * a + ROUND[typ] * np.abs(ref)
        assert np.all(np.abs(got[i] - ref) <= bound), (i, p)


# ---------------------------------------------------------------- a strong key with a small value

LOW, HIGH = 127 * 2.0 ** -12, 127 * 2.0 ** -5


@functools.lru_cache
def sink_batch(value, dim, weak):
    """1400 tokens of which one, in the middle, has a key of HIGH throughout and values of size `value`; the others' are LOW
    and `weak`.  The keys' codes and scales are exact, so is d * q in 11 bits: the scores carry no error of the cached
    numbers."""
    rng = np.random.default_rng(1020)
    batch = kp.make([1400], [1], 1, dim, 64, rng)
    for p in range(1400):
        v = rng.standard_normal((1, dim)).astype(np.float32)
        key, size = (HIGH, value) if p == 700 else (LOW, weak)
        kp.write(batch, 0, p, np.full((1, dim), key, np.float32), v * np.float32(size))
    return batch


SINK = [(typ, dim, n) for typ, dim in (("f32", 64), ("f32", 128), ("f32", 256), ("bf16", 64), ("bf16", 128), ("bf16", 256), ("f16", 128))
        for n in (1, 5)] + [("f32", 256, 80)]
SINK += [("f32", 64, 80), ("f32", 128, 80)]
SINK += [("bf16", 64, 80), ("bf16", 128, 80), ("bf16", 256, 80), ("f16", 128, 80)]


@pytest.mark.parametrize("typ,dim,n", SINK)
@pytest.mark.parametrize("gap", [14.0, 18.0, 24.0, 45.0])
@pytest.mark.parametrize("value", [0.0, 1e-4])
def test_a_strong_key_with_a_small_value(value, gap, typ, dim, n):
    """The weak keys make the result where the strong one's value is small, however small their weights are: held to the
    2-norm of the type (f32: 1e-5; 16 bits: values and probabilities of 11 bits, together 2^-10, and the result's rounding,
    or half its smallest number)."""
    if typ == "f16" and gap > 24.0:
        gap = 20.0
    batch = sink_batch(value, dim, 1.0 if typ == "f32" else 8000.0)  # so that f16 holds the result
    batch.counts = [n]
    scale = float(gap / (dim * (HIGH - LOW)))
    q, qh = token_array(np.ones((n, 2, dim), np.float32), typ)
    got = attend(batch, q, typ, 2, scale)
    for i in {*range(0, n, 11), n - 1}:
        ref, _ = row_attention(batch, 0, qh[i], 0, 1400 - n + i + 1, scale)
        err = np.linalg.norm(got[i] - ref)
        tol = 1e-5 if typ == "f32" else 2.0 ** -10 + ROUND[typ]
        floor = 2.0 ** -25 * np.sqrt(ref.size) if typ == "f16" else 0.0
        assert err <= tol * np.linalg.norm(ref) + floor, (i, err / np.linalg.norm(ref))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 80])
@pytest.mark.parametrize("first", [0, 60, 300])
def test_whole_tiles_without_values(first, n, typ):
    """Tokens `first` .. `first` + 299 have values of 0, and among them is the strong key."""
    rng = np.random.default_rng(1022)
    kv, dim, gap = 900, 64, 24.0
    batch = kp.make([kv], [n], 1, dim, 64, rng)
    for p in range(kv):
        key = HIGH if p == first + 130 else LOW
        v = rng.standard_normal((1, dim)) * (0.0 if first <= p < first + 300 else 1.0)
        kp.write(batch, 0, p, np.full((1, dim), key, np.float32), v.astype(np.float32))
    q, qh = token_array(np.ones((n, 2, dim), np.float32), typ)
    scale = float(gap / (dim * (HIGH - LOW)))
    got = attend(batch, q, typ, 2, scale)
    for i in {*range(0, n, 11), n - 1}:
        ref, _ = row_attention(batch, 0, qh[i], 0, kv - n + i + 1, scale)
        tol = 1e-5 if typ == "f32" else 2.0 ** -10 + ROUND[typ]
        assert np.linalg.norm(got[i] - ref) <= tol * np.linalg.norm(ref), (i, np.linalg.norm(got[i] - ref) / np.linalg.norm(ref))


ANYWHERE = [("f32", 1), ("bf16", 1)]
ANYWHERE += [("f32", 200)]
ANYWHERE += [("bf16", 200), ("f16", 200)]


@pytest.mark.parametrize("typ,n", ANYWHERE)
def test_strong_keys_with_small_values_anywhere(typ, n):
    """Several of them, in several tiles, seen by some rows only, with a window; values of one token many orders apart
    from the next one's elsewhere."""
    rng = np.random.default_rng(1021)
    kv, dim, heads = 900, 128, 4
    batch = kp.make([kv], [n], 2, dim, 16, rng, fill=0xFF)
    strong = set(rng.choice(kv, 12, replace=False).tolist()) | {kv - 60, 0}
    for p in range(kv):
        k = rng.standard_normal((2, dim)).astype(np.float32) * np.float32(0.25)
        v = rng.standard_normal((2, dim)).astype(np.float32)
        if p in strong:
            k = k + np.float32(1.0)
            v = v * np.float32(10.0 ** rng.integers(-7, -3))
        elif p % 13 == 0:
            v = v * np.float32(10.0 ** rng.integers(-3, 3))
        kp.write(batch, 0, p, k, v)
    q = (np.full((n, heads, dim), 1.0) + rng.standard_normal((n, heads, dim)) * 0.3).astype(np.float32)
    for window in (0, 333):
        check_attention(batch, heads, typ, rng, q=q, window=window, norm=typ == "f32")


# ---------------------------------------------------------------- scores of any size

SCORES = [(typ, dim, n, scale) for typ, dim in (("f32", 64), ("f32", 256), ("bf16", 64), ("bf16", 256), ("f16", 128))
          for n in (1, 6) for scale in (50.0, 1e3, 1e4, 1e5, 1e7, 1e28)]
SCORES += [("f32", 256, 80, 1e28)]
# the chunk kernels: scores up to 2^19, the stated range
SCORES += [("f32", 64, 80, 50.0), ("f32", 128, 80, 50.0), ("bf16", 64, 80, 50.0), ("bf16", 256, 80, 50.0), ("f16", 128, 80, 50.0)]


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("typ,dim,n,scale", SCORES)
def test_scores_of_any_size(typ, dim, n, scale, sign):
    """One visible key counts whatever its score (down to -1e32 here), and of several the one with the largest."""
    rng = np.random.default_rng(1030)
    kv = 100
    batch = kp.make([kv], [n], 1, dim, 16, rng)
    for p in range(kv):
        kp.write(batch, 0, p, np.full((1, dim), 1.0 + 0.125 * (p * 7 % 11), np.float32), rng.standard_normal((1, dim)).astype(np.float32))
    q, qh = token_array(np.full((n, 2, dim), sign * 4096.0 / dim, np.float32), typ)
    for window in (1, 3, 9, 0):
        got = attend(batch, q, typ, 2, scale, window=window)
        for i in {*range(0, n, 7), n - 1}:
            p = kv - n + i
            lo = max(0, p - window + 1) if window else 0
            ref, _ = row_attention(batch, 0, qh[i], lo, p + 1, scale)
            # equal scores among the visible keys are equal sums of equal products: their mean, by the type's rounding
            assert np.linalg.norm(got[i] - ref) <= (1e-5 if typ == "f32" else 2.0 ** -10 + ROUND[typ]) * np.linalg.norm(ref), (window, i)



# ---------------------------------------------------------------- soft-caps
@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 80])
@pytest.mark.parametrize("cap", [1e-44, 1e-39, 1e-30, 1e30])
def test_soft_caps_of_any_size(cap, n, typ):
    """A tiny cap makes every score 0 (the mean of the visible values, a score of exactly 0 included), a huge one none."""
    rng = np.random.default_rng(1031)
    batch = random_batch([120], [n], 1, 64, 16, rng)
    q = rng.standard_normal((n, 2, 64)).astype(np.float32)
    q[:, 1] = 0.0  # scores of exactly 0
    q, qh = token_array(q, typ)
    got = attend(batch, q, typ, 2, 0.125, softcap=cap)
    for i in range(n):
        ref, a = row_attention(batch, 0, qh[i], 0, 120 - n + i + 1, 0.125 if cap > 1 else 0.0)
        bound = (2.1 * 2.0 ** -16 + 2.0 ** -16) * a if typ == "f32" else (2.1 * 2.0 ** -6 + 2.0 ** -10) * a + ROUND[typ] * np.abs(ref)
        assert np.all(np.abs(got[i] - ref) <= bound), i


# ---------------------------------------------------------------- the scale

def test_the_scale_is_the_rounded_quotient():
    """d = fp16(max|x| / 127), the quotient rounded to f32 as in the library's quantizer.  Next to a tie of the fp16
    rounding a product with a rounded 1 / 127 gives another scale: at these magnitudes, found by trying all."""
    near = np.array([float.fromhex(x) for x in ("0x1.fc3f82p+0", "0x1.fd3d82p+0", "0x1.fe3b82p+0", "0x1.ff3982p+0")], np.float32)
    amax = np.concatenate([near * np.float32(2.0 ** e) for e in (-8, -1, 0, 3, 11)] + [np.float32([1e-30, 6e4, 3e38, 127.0, 1.0])])
    rng = np.random.default_rng(1040)
    n, dim = len(amax), 64
    x = (rng.uniform(-1, 1, (n, dim)) * amax[:, None]).astype(np.float32)
    x[:, 5] = amax
    x[:, 40] = -amax
    batch = kp.make([n], [n], 1, dim, 16, rng)
    xd = dev(x)
    cache = dev(batch.cache)
    gq.gq_kv_append_q8_0(xd, dim, xd, dim, gq.GQ_TYPE_F32, cache, *lists(batch), *sizes(batch))
    raw = cache.cpu().numpy()
    kc, ks, vc, vs = kp.layout(dim)
    want = np.minimum(amax / np.float32(127), np.float32(515.5)).astype(np.float16)
    for p in range(n):
        pg, rec, tk = batch.record(0, p)
        r = raw[pg, 0, rec]
        d = want[p].astype(np.float32)
        y = x[p] / d if d > 0 else np.zeros(dim, np.float32)
        code = np.clip(np.sign(y) * np.floor(np.abs(y.astype(np.float64)) + 0.5), -127, 127)
        for c, s in ((kc, ks), (vc, vs)):
            got = (r[s[tk]].astype(np.uint16) | (r[s[tk] + 1].astype(np.uint16) << 8)).view(np.float16)
            assert np.array_equal(got, np.repeat(want[p], 2)), (p, amax[p], got, want[p])
            assert np.array_equal(r[c[tk]].astype(np.int64) - 128, code), p


# ---------------------------------------------------------------- nothing to do

def test_calls_without_tokens_take_empty_arrays():
    """n_tokens = 0 does nothing, also where the token arrays are empty tensors (whose address is null)."""
    t = torch()
    rng = np.random.default_rng(1050)
    batch = random_batch([20], [0], 1, 64, 16, rng)
    cache = dev(batch.cache)
    x = t.empty((0, 64), device="cuda")
    ws = t.zeros(gq.gq_kv_attention_workspace_bytes(1, 1, 64), dtype=t.uint8, device="cuda")
    gq.gq_kv_append_q8_0(x, 64, x, 64, gq.GQ_TYPE_F32, cache, *lists(batch), *sizes(batch))
    gq.gq_kv_read_q8_0(cache, *lists(batch), x, 64, x, 64, gq.GQ_TYPE_F32, *sizes(batch))
    gq.gq_kv_attention_q8_0(x, 64, cache, *lists(batch), x, 64, gq.GQ_TYPE_F32, 1.0, 0.0, 0, ws, ws.numel(), 1, *sizes(batch))
    assert np.array_equal(cache.cpu().numpy(), batch.cache)
    assert gq.gq_device_status() == gq.GQ_OK
