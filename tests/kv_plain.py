"""Plain numpy forms of the paged Q8_0 cache and its attention, in 64 bits.

The record layout is written here from its description in include/gq_kv.h,
byte by byte, and shares no code with the kernels or the benchmark."""

from __future__ import annotations

import dataclasses

import numpy as np

REC = 16


def layout(dim):
    """Byte offsets inside a record: K codes [16][dim], K scales [16][nb], V codes [16][dim], V scales [16][nb]."""
    nb = dim // 32
    kc = np.empty((REC, dim), np.int64)
    ks = np.empty((REC, nb), np.int64)
    vc = np.empty((REC, dim), np.int64)
    vs = np.empty((REC, nb), np.int64)
    for t in range(REC):
        key = (t & 1) + 2 * ((t // 4) % 2) if nb > 2 else (t // 4) % 2
        for e in range(dim):
            b = e // 32
            kc[t, e] = 32 * (t * nb + (b ^ key)) + e % 32
            g = t // 4
            vc[t, e] = 17 * dim + g * 4 * dim + 16 * ((e // 4) ^ (2 * g)) + 4 * (e % 4) + t % 4
        for b in range(nb):
            ks[t, b] = 16 * dim + 2 * (t * nb + b)
            vs[t, b] = 33 * dim + 2 * (b * REC + t)
    return kc, ks, vc, vs


def quantise(x):
    """[..., dim] f32 -> (codes int, scales f16): the rule of gq_kv_append_q8_0."""
    x = np.asarray(x, np.float32)
    x = x.reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(over="ignore", invalid="ignore"):
        amax = np.fmax.reduce(np.abs(x), axis=-1, initial=np.float32(0))
        d = np.minimum(amax * (np.float32(1) / np.float32(127)), np.float32(515.5)).astype(np.float16)
        df = d.astype(np.float32)[..., None]
        y = np.divide(x, df, out=np.zeros_like(x), where=df > 0)
        q = np.sign(y) * np.floor(np.abs(y.astype(np.float64)) + 0.5)
    q = np.where(np.isnan(y), -127.0, np.clip(q, -127, 127))
    q = np.where(df > 0, q, 0.0).astype(np.int64)
    return q.reshape(q.shape[:-2] + (-1,)), d


@dataclasses.dataclass
class Batch:
    """A batch with its host lists and its cache as bytes [page][head][record][34 dim]."""
    kv_len: list
    counts: list
    kv_heads: int
    dim: int
    page: int
    table: np.ndarray
    cache: np.ndarray

    @property
    def starts(self):
        return np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)

    @property
    def n_tokens(self):
        return int(sum(self.counts))

    def positions(self, b):
        return range(self.kv_len[b] - self.counts[b], self.kv_len[b])

    def record(self, b, pos):
        return self.table[b, pos // self.page], pos % self.page // REC, pos % REC


def make(kv_len, counts, kv_heads, dim, page, rng, spare=2, fill=0):
    """An empty cache with pages handed out in random order; table entries past a sequence's pages are -1."""
    need = [-(-kv // page) for kv in kv_len]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages)
    table = np.full((len(kv_len), max(1, max(need)) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = np.full((n_pages, kv_heads, page // REC, 34 * dim), fill, np.uint8)
    return Batch(list(kv_len), list(counts), kv_heads, dim, page, table, cache)


def write(batch, b, pos, k, v):
    """Store one token's keys and values ([heads][dim] f32) at a position."""
    kc, ks, vc, vs = layout(batch.dim)
    pg, rec, t = batch.record(b, pos)
    out = batch.cache[pg, :, rec]
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        q, d = quantise(x)
        out[:, c[t]] = ((q + 128) & 255).astype(np.uint8)
        raw = d.view(np.uint16)
        out[:, s[t]] = (raw & 255).astype(np.uint8)
        out[:, s[t] + 1] = (raw >> 8).astype(np.uint8)


def values(batch, b, pos):
    """K and V of the positions `pos` of sequence b: f64 [len(pos)][heads][dim]."""
    kc, ks, vc, vs = layout(batch.dim)
    pos = np.asarray(list(pos), np.int64)
    if not len(pos):
        z = np.zeros((0, batch.kv_heads, batch.dim))
        return z, z
    raw = batch.cache[batch.table[b][pos // batch.page], :, pos % batch.page // REC].astype(np.int64)  # [n][heads][bytes]
    t = pos % REC
    got = []
    for c, s in ((kc, ks), (vc, vs)):
        code = np.take_along_axis(raw, np.broadcast_to(c[t][:, None, :], raw.shape[:2] + (batch.dim,)), -1) - 128
        at = np.broadcast_to(s[t][:, None, :], raw.shape[:2] + (batch.dim // 32,))
        d = np.take_along_axis(raw, at, -1) + 256 * np.take_along_axis(raw, at + 1, -1)
        d = d.astype(np.uint16).view(np.float16).astype(np.float64)
        got.append(code * np.repeat(d, 32, axis=-1))
    return got


def attention(batch, q, scale, softcap=0.0, window=0):
    """(o, sum w |v|, largest scale * sum |q k| over the visible keys), f64 [n_tokens][heads][dim] (the last [n_tokens][heads])."""
    heads = q.shape[1]
    group = heads // batch.kv_heads
    o = np.zeros(q.shape)
    a = np.zeros(q.shape)
    mag = np.zeros(q.shape[:2])
    for b in range(len(batch.kv_len)):
        k, v = values(batch, b, range(batch.kv_len[b]))
        for i, p in enumerate(batch.positions(b)):
            row = batch.starts[b] + i
            lo = max(0, p - window + 1) if window else 0
            if p < lo:
                continue
            for h in range(heads):
                kk, vv = k[lo:p + 1, h // group], v[lo:p + 1, h // group]
                s = scale * (kk @ q[row, h].astype(np.float64))
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                w = np.exp(s - s.max())
                w /= w.sum()
                o[row, h] = w @ vv
                a[row, h] = w @ np.abs(vv)
                mag[row, h] = abs(scale) * (np.abs(kk) @ np.abs(q[row, h].astype(np.float64))).max()
    return o, a, mag
