"""Workloads of the paged Q8_0 key/value cache and the attention that reads it.

Three operators: `append` (quantise new keys and values into the cache),
`read` (give them back in a floating type) and `attention` (new tokens
against the cached ones; one new token a sequence is its decode form).

The cache is an array of pages of `page` tokens.  A page holds, for every kv
head, one record per 16 tokens of 34 * dim bytes:

    16 * dim   K codes: token t, 32-block b at 32-byte unit t * nb + (b ^ key(t)),
               byte = code + 128
    dim        K scales, f16 [16 tokens][nb]
    16 * dim   V codes: for each group of four tokens, one 4-byte word per
               element d holding the four tokens' bytes (code + 128); 16-byte
               chunk d / 4 of group g sits at chunk (d / 4) ^ (2 g)
    dim        V scales, f16 [nb][16 tokens]

with nb = dim / 32 and key(t) = (t & 1) | (t >> 1 & 2), or t >> 2 & 1 for nb = 2.

New tokens of sequence b are rows q_start[b] .. q_start[b + 1] of the inputs
and occupy the last positions of its kv_len[b] cached ones.
"""

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- cases

def listed():
    base = {"heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "softcap": 0.0, "spread": 1.0, "fused": False}

    def case(name, **kw):
        return dict(base, name=name, **kw)

    return [
        # one user's next token: the smallest write, all latency
        case("append_1x1_f32", op="append", type="f32", n_seq=1, q=1, kv=200, fused=True),
        # a serving batch's next tokens, written from the fused projection's rows
        case("append_64x1_bf16", op="append", type="bf16", n_seq=64, q=1, kv=700, page=16, spread=0.3, fused=True),
        # prompts of odd lengths, written whole, in the projections' own f32
        case("append_prompts_f32", op="append", type="f32", n_seq=6, q=4099, kv=4099, spread=0.4),
        # a short cached prefix read back for a consumer in f32
        case("read_1x333_f32", op="read", type="f32", n_seq=1, q=333, kv=333),
        # a batch of contexts moved out of the pages in 16 bits
        case("read_8x8192_bf16", op="read", type="bf16", n_seq=8, q=8192, kv=8192, spread=0.7, page=128),
        # one token of one short conversation: latency
        case("decode_1x129_f32", op="attention", type="f32", n_seq=1, q=1, kv=129, page=16, fused=True),
        # one token of one long context: the work has to be split along the keys
        case("decode_1x131072_bf16", op="attention", type="bf16", n_seq=1, q=1, kv=131072),
        # a serving batch of ragged contexts, wide heads, a score soft-cap
        case("decode_48x9000_f32", op="attention", type="f32", n_seq=48, q=1, kv=9000, heads=16, dim=256, spread=0.15,
             softcap=50.0, page=32),
        # five drafted tokens a sequence, one head a group, a sliding window
        case("verify_16x5_window_bf16", op="attention", type="bf16", n_seq=16, q=5, kv=5000, heads=16, kv_heads=16,
             spread=0.5, window=1024, page=16),
        # a chunk of a prompt behind a long cached prefix, in the framework's f32
        case("chunk_509_of_8191_f32", op="attention", type="f32", n_seq=1, q=509, kv=8191, fused=True),
        # prompts of odd lengths in one call, narrow heads in groups of five
        case("chunk_7_prompts_f16", op="attention", type="f16", n_seq=7, q=1213, kv=1900, heads=20, kv_heads=4, dim=64,
             spread=0.2, page=16),
        # the largest: a full prefill chunk behind a long prefix
        case("chunk_2048_of_32768_bf16", op="attention", type="bf16", n_seq=1, q=2048, kv=32768, page=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "attention"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    dim = rng.choice([64, 128, 128, 256])
    case = {"op": op, "type": rng.choice(["f32", "bf16", "f16"]), "kv_heads": kv_heads,
            "heads": kv_heads * min(rng.choice([1, 2, 4, 5, 7, 8, 16]), 64 // kv_heads), "dim": dim, "page": rng.choice([16, 32, 64, 128]),
            "window": 0, "softcap": 0.0, "spread": round(rng.uniform(0.1, 1.0), 3), "fused": rng.random() < 0.5}
    if op != "attention":
        n_seq = _log_int(rng, 1, 64)
        # at most what the largest read moves: 64 Mi elements of K
        most = max(1, min(16384, (1 << 26) // (n_seq * kv_heads * dim)))
        q = _log_int(rng, 1, most)
        return dict(case, n_seq=n_seq, q=q, kv=q + (_log_int(rng, 1, 500) if op == "append" else 0))
    if rng.random() < 0.25:
        case["softcap"] = rng.choice([20.0, 50.0])
    n_seq = _log_int(rng, 1, 64)
    q = 1 if rng.random() < 0.5 else _log_int(rng, 2, 2048)
    n_seq = min(n_seq, max(1, 4096 // q))
    # bounded by the largest listed case's scores and by 64 Mi elements of K
    most = min(131072, (1 << 29) // (n_seq * q * case["heads"]), (1 << 27) // (n_seq * kv_heads * dim))
    kv = max(q, _log_int(rng, min(64, most), most))
    if rng.random() < 0.25:
        case["window"] = _log_int(rng, 16, 4096)
    return dict(case, n_seq=n_seq, q=q, kv=kv)


def _lengths(case):
    """(new tokens, cached tokens) of every sequence: spread over [spread, 1] times the largest, the largest first."""
    got = []
    for b in range(case["n_seq"]):
        f = 1.0 - (1.0 - case["spread"]) * ((b * 0.6180339887498949) % 1.0)
        g = 1.0 - (1.0 - case["spread"]) * ((b * 0.7548776662466927) % 1.0)
        n = max(1, int(case["q"] * f))
        got.append((n, max(n, int(case["kv"] * (f if case["op"] == "read" else g)))))
    return got


def _visible(case):
    """(query-key pairs, cached tokens that some query sees), summed over the sequences."""
    pairs = tokens = 0
    for n, kv in _lengths(case):
        w = case["window"] or kv
        first = kv - n
        short = min(n, max(0, w - 1 - first))  # the queries with fewer than w positions up to their own
        pairs += (first + 1 + first + short) * short // 2 + (n - short) * w
        tokens += kv - max(0, first - w + 1)
    return pairs, tokens


def work(case):
    el, d = _SIZE[case["type"]], case["dim"]
    n = sum(x for x, _ in _lengths(case))
    if case["op"] != "attention":
        # each new key and value once in its type and once as codes with scales; about ten operations an element
        return {"bytes": 2 * n * case["kv_heads"] * d * (el + 34 / 32), "flops": 20 * n * case["kv_heads"] * d}
    pairs, tokens = _visible(case)
    return {"bytes": tokens * case["kv_heads"] * d * 2 * 34 / 32 + 2 * n * case["heads"] * d * el + 4 * case["n_seq"],
            "flops": 4 * d * case["heads"] * pairs}


# ---------------------------------------------------------------- layout

def _k_order(nb, device):
    """[16][nb]: where block b of token t sits among the token's units."""
    t = torch.arange(16, device=device)
    key = (t & 1) | (t >> 1 & 2) if nb > 2 else t >> 2 & 1
    return torch.arange(nb, device=device)[None, :] ^ key[:, None]


def _v_order(dim, device):
    """[4][dim / 4]: where chunk c of token group g sits among the group's chunks."""
    return torch.arange(dim // 4, device=device)[None, :] ^ (2 * torch.arange(4, device=device)[:, None])


def _planes(cache, case):
    """Views of the cache: K codes [page][head][record][16][nb][32], K scales [...][16][nb], V codes
    [...][4][dim / 4][4 elements][4 tokens], V scales [...][nb][16]."""
    d, nb = case["dim"], case["dim"] // 32
    rec = cache.view(-1, case["kv_heads"], case["page"] // 16, 34 * d)
    return (rec[..., :16 * d].unflatten(-1, (16, nb, 32)), rec[..., 16 * d:17 * d].view(torch.float16).unflatten(-1, (16, nb)),
            rec[..., 17 * d:33 * d].unflatten(-1, (4, d // 4, 4, 4)), rec[..., 33 * d:].view(torch.float16).unflatten(-1, (nb, 16)))


def _quantise(x):
    """[..., nb, 32] -> (byte codes, f16 scales), in 32 bits."""
    x = x.float()
    d = torch.clamp(x.abs().amax(-1) / 127.0, max=515.5).half()
    df = d.float()[..., None]
    y = (x / torch.where(df > 0, df, 1.0)).abs()
    whole = torch.trunc(y)
    whole = torch.clamp(whole + ((y - whole) >= 0.5).float(), max=127.0)
    code = torch.where(df > 0, torch.where(x < 0, -whole, whole), 0.0)
    return (code + 128.0).to(torch.uint8), d


def _positions(state):
    """(sequence, position) of every new token."""
    q_start = state["q_start"].long()
    row = torch.arange(state["n_tokens"], device=q_start.device)
    seq = torch.searchsorted(q_start[1:].contiguous(), row, right=True)
    return seq, state["kv_len"].long()[seq] - q_start[seq + 1] + row


# ---------------------------------------------------------------- what a user has in hand

def prepare(case, seed):
    case = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, nb, hk, hq, page = case["dim"], case["dim"] // 32, case["kv_heads"], case["heads"], case["page"]
    typ = _TYPES[case["type"]]
    lens = _lengths(case)
    max_pages = max(-(-kv // page) for _, kv in lens)
    used = sum(-(-kv // page) for _, kv in lens)
    n_pages = used + 3
    # pages handed out in no order, as after a while of serving; entries past a sequence's pages are never read
    order = torch.randperm(n_pages, generator=g, device="cuda")[:used].to(torch.int32)
    count = torch.tensor([-(-kv // page) for _, kv in lens], device="cuda")
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_pages, device="cuda")[None, :] < count[:, None]] = order
    n_tokens = sum(n for n, _ in lens)
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    state = {"case": case, "table": table, "n_tokens": n_tokens, "n_pages": n_pages, "max_pages": max_pages,
             "max_q": max(n for n, _ in lens), "max_kv": max(kv for _, kv in lens),
             "kv_len": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
             "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda")}
    # the cache as earlier tokens left it: keys with a few strong channels, values without
    cache = torch.zeros(n_pages * hk * (page // 16) * 34 * d, dtype=torch.uint8, device="cuda")
    if case["op"] != "append":
        kc, ks, vc, vs = _planes(cache, case)
        strong = 1.0 + 3.0 * (torch.rand(nb, 32, generator=g, device="cuda") < 0.04)
        step = max(1, (1 << 25) // (hk * page * d))
        at = torch.arange(16, device="cuda")[:, None], _k_order(nb, "cuda")
        vat = torch.arange(4, device="cuda")[:, None], _v_order(d, "cuda")
        for p in range(0, n_pages, step):
            n = min(step, n_pages - p)
            x = torch.randn(n, hk, page // 16, 16, nb, 32, generator=g, device="cuda") * strong
            code, scale = _quantise(x)
            kc[p:p + n, :, :, at[0], at[1]] = code
            ks[p:p + n] = scale
            x = torch.randn(n, hk, page // 16, 16, nb, 32, generator=g, device="cuda")
            code, scale = _quantise(x)
            vc[p:p + n, :, :, vat[0], vat[1]] = code.reshape(n, hk, page // 16, 4, 4, d // 4, 4).permute(0, 1, 2, 3, 5, 6, 4)
            vs[p:p + n] = scale.transpose(-1, -2)
    state["cache"] = cache
    if case["op"] == "append":
        state["written"] = dict(zip(("k_codes", "k_scales", "v_codes", "v_scales"), _planes(cache, case)))
    # the new tokens' rows: q, k and v of a token side by side where one projection made them, with its padding
    width = (hq + 2 * hk) * d + 64
    x = torch.randn(n_tokens, width, generator=g, device="cuda")
    x[:, :hq * d] *= 2.0
    x = x.to(typ)
    parts = [x[:, :hq * d], x[:, hq * d:(hq + hk) * d], x[:, (hq + hk) * d:(hq + 2 * hk) * d]]
    if not case["fused"]:
        parts = [p.contiguous() for p in parts]
    need = {"append": ("k", "v"), "read": (), "attention": ("q",)}[case["op"]]
    state.update({n: p for n, p in zip("qkv", parts) if n in need})
    if case["op"] == "read":
        state["k"] = torch.empty(n_tokens, hk * d, dtype=typ, device="cuda")
        state["v"] = torch.empty(n_tokens, hk * d, dtype=typ, device="cuda")
    if case["op"] == "attention":
        state["out"] = torch.empty(n_tokens, hq * d, dtype=typ, device="cuda")
    return state


# ---------------------------------------------------------------- plain forms

def _plain_append(state):
    case = state["case"]
    nb, hk, d = case["dim"] // 32, case["kv_heads"], case["dim"]
    n = state["n_tokens"]
    seq, pos = _positions(state)
    page, rec, tok = state["table"].long()[seq, pos // case["page"]], pos % case["page"] // 16, pos % 16
    kc, ks, vc, vs = _planes(state["cache"], case)
    head = torch.arange(hk, device=page.device)[None, :, None]
    code, scale = _quantise(state["k"].reshape(n, hk, nb, 32))
    at = page[:, None, None], head, rec[:, None, None], tok[:, None, None]
    kc[at + (_k_order(nb, page.device)[tok][:, None, :],)] = code
    ks[at + (torch.arange(nb, device=page.device)[None, None, :],)] = scale
    code, scale = _quantise(state["v"].reshape(n, hk, nb, 32))
    chunk = _v_order(d, page.device)[tok // 4][:, None, :, None]
    vc[page[:, None, None, None], head[..., None], rec[:, None, None, None], tok[:, None, None, None] // 4, chunk,
       torch.arange(4, device=page.device), tok[:, None, None, None] % 4] = code.reshape(n, hk, d // 4, 4)
    vs[at[:3] + (torch.arange(nb, device=page.device)[None, None, :], at[3])] = scale
    return state["written"]


def _values(planes, case):
    """K and V of whole records in 32 bits: [...][16][dim] each."""
    kc, ks, vc, vs = planes
    d, nb = case["dim"], case["dim"] // 32
    dev = kc.device
    k = kc[..., torch.arange(16, device=dev)[:, None], _k_order(nb, dev), :].float() - 128.0
    v = vc[..., torch.arange(4, device=dev)[:, None], _v_order(d, dev), :, :].float() - 128.0
    k = (k * ks.float()[..., None]).flatten(-2)
    v = v.flatten(-3, -2).transpose(-1, -2).flatten(-3, -2).unflatten(-1, (nb, 32))
    return k, (v * vs.float().transpose(-1, -2)[..., None]).flatten(-2)


def _cached(state):
    """Every sequence's cached K and V in 32 bits, [seq][head][token][dim], up to the longest."""
    planes = [p[state["table"].long().clamp(min=0)] for p in _planes(state["cache"], state["case"])]
    return [x.permute(0, 2, 1, 3, 4, 5).flatten(2, 4)[:, :, :state["max_kv"]] for x in _values(planes, state["case"])]


def _plain_read(state):
    seq, pos = _positions(state)
    typ = _TYPES[state["case"]["type"]]
    k, v = _cached(state)
    return {"k": k[seq, :, pos].flatten(1).to(typ), "v": v[seq, :, pos].flatten(1).to(typ)}


def _plain_attention(state):
    case = state["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    n_seq, mq, mkv, grp = case["n_seq"], state["max_q"], state["max_kv"], hq // hk
    k, v = _cached(state)
    q_start, kv_len = state["q_start"].long(), state["kv_len"].long()
    count = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=k.device)
    row = (q_start[:-1, None] + i[None, :]).clamp(max=state["n_tokens"] - 1)
    q = state["q"].reshape(state["n_tokens"], hk, grp, d)[row].float()    # [seq][q][head][group][dim]
    q = q.permute(0, 2, 1, 3, 4).reshape(n_seq, hk, mq * grp, d)
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    if case["softcap"] > 0:
        s = (s / case["softcap"]).tanh_().mul_(case["softcap"])
    p = (kv_len - count)[:, None] + i[None, :]                            # position of every query
    j = torch.arange(mkv, device=k.device)
    hidden = (j[None, None, :] > p[:, :, None])
    if case["window"]:
        hidden |= j[None, None, :] <= p[:, :, None] - case["window"]
    s.view(n_seq, hk, mq, grp, mkv).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s @ v) / torch.where(total > 0, total, 1.0)
    o = o.view(n_seq, hk, mq, grp, d).permute(0, 2, 1, 3, 4).reshape(n_seq, mq, hq * d)
    return o[i[None, :] < count[:, None]].to(_TYPES[case["type"]])


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention}[case["op"]](state)
    import block_quantized_matvec_gq_gb300 as gq

    typ = {"f32": gq.GQ_TYPE_F32, "bf16": gq.GQ_TYPE_BF16, "f16": gq.GQ_TYPE_F16}[case["type"]]
    sizes = (state["n_pages"], state["max_pages"], case["page"], case["kv_heads"], case["dim"], case["n_seq"], state["n_tokens"])
    lists = (state["table"], state["kv_len"], state["q_start"])
    if case["op"] == "append":
        k, v = state["k"], state["v"]
        gq.gq_kv_append_q8_0(k, k.stride(0), v, v.stride(0), typ, state["cache"], *lists, *sizes)
        return state["written"]
    if case["op"] == "read":
        k, v = state["k"], state["v"]
        gq.gq_kv_read_q8_0(state["cache"], *lists, k, k.stride(0), v, v.stride(0), typ, *sizes)
        return {"k": k, "v": v}
    if "workspace" not in state:  # kept by the program, zero-filled once
        n = gq.gq_kv_attention_workspace_bytes(case["heads"], case["kv_heads"], case["dim"])
        state["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    q, out, ws = state["q"], state["out"], state["workspace"]
    gq.gq_kv_attention_q8_0(q, q.stride(0), state["cache"], *lists, out, out.stride(0), typ, 1.0 / math.sqrt(case["dim"]),
                            case["softcap"], case["window"], ws, ws.numel(), case["heads"], *sizes)
    return out


# ---------------------------------------------------------------- the definition in 64 bits

def _record(raw, dim):
    """One head's records of one page, bytes [records][34 * dim] -> K and V [16 * records][dim] in 64 bits."""
    n, nb = raw.shape[0], dim // 32
    t = torch.arange(16, device=raw.device)[:, None]
    e = torch.arange(dim, device=raw.device)[None, :]
    key = (t & 1) + 2 * ((t >> 2) & 1) if nb > 2 else (t >> 2) & 1
    k_byte = 32 * (t * nb + ((e // 32) ^ key)) + e % 32
    v_byte = 17 * dim + (t // 4) * 4 * dim + 16 * ((e // 4) ^ (2 * (t // 4))) + 4 * (e % 4) + t % 4
    k_scale = raw[:, 16 * dim:17 * dim].contiguous().view(torch.float16).double()[:, t * nb + e // 32]
    v_scale = raw[:, 33 * dim:].contiguous().view(torch.float16).double()[:, (e // 32) * 16 + t]
    k = (raw[:, k_byte].double() - 128) * k_scale
    v = (raw[:, v_byte].double() - 128) * v_scale
    return k.reshape(16 * n, dim), v.reshape(16 * n, dim)


def exact(case, seed):
    state = prepare(case, seed)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens = _lengths(case)
    if case["op"] == "append":
        # the codes are whole numbers; a scale stands for amax / 127
        _, ks, _, vs = _planes(state["cache"], case)
        ks, vs = ks.double(), vs.double()
        for name, out in (("k", ks), ("v", vs)):
            scale = state[name].double().reshape(state["n_tokens"], hk, d // 32, 32).abs().amax(-1) / 127
            for b, (n, kv) in enumerate(lens):
                r0 = int(state["q_start"][b])
                pos = torch.arange(kv - n, kv, device="cuda")
                pg = state["table"][b].long()[pos // page]
                if name == "k":
                    out[pg, :, pos % page // 16, pos % 16] = scale[r0:r0 + n]
                else:
                    out[pg, :, pos % page // 16, :, pos % 16] = scale[r0:r0 + n]
        return {"k_codes": None, "k_scales": ks, "v_codes": None, "v_scales": vs}
    raw = state["cache"].view(state["n_pages"], hk, page // 16, 34 * d)
    outs = []
    for b, (n, kv) in enumerate(lens):
        pages = state["table"][b, :-(-kv // page)].long()
        heads = []
        for h in range(hk):
            k, v = _record(raw[pages, h].reshape(-1, 34 * d), d)
            k, v = k[:kv], v[:kv]
            if case["op"] == "read":
                heads.append((k[kv - n:], v[kv - n:]))
                continue
            r0 = int(state["q_start"][b])
            q = state["q"][r0:r0 + n].double().reshape(n, hk, hq // hk, d)[:, h]
            pos = torch.arange(kv - n, kv, device="cuda")
            part = []
            step = max(1, (1 << 27) // (kv * (hq // hk)))
            for a in range(0, n, step):
                s = torch.einsum("qgd,kd->qgk", q[a:a + step], k) / math.sqrt(d)
                if case["softcap"] > 0:
                    s = case["softcap"] * torch.tanh(s / case["softcap"])
                j = torch.arange(kv, device="cuda")
                seen = j <= pos[a:a + step, None]
                if case["window"]:
                    seen &= j > pos[a:a + step, None] - case["window"]
                w = torch.softmax(s.masked_fill(~seen[:, None, :], -math.inf), -1)
                part.append(torch.einsum("qgk,kd->qgd", w, v))
            heads.append(torch.cat(part))
        if case["op"] == "read":
            outs.append(tuple(torch.stack(x, 1).reshape(n, hk * d) for x in zip(*heads)))
        else:
            outs.append(torch.stack(heads, 1).reshape(n, hq * d))
    if case["op"] == "read":
        return {"k": torch.cat([x for x, _ in outs]), "v": torch.cat([x for _, x in outs])}
    return torch.cat(outs)
