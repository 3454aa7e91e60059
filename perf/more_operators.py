"""Workloads of what a serving step does around the projections and the attention.

Four operators, in the order of a step:

`plan`    the batch's lists from the requests' lengths: pages handed out and taken
          back, the block table, q_start, kv_len, and every new token's slot,
          position and sequence;
`embed`   the new tokens' rows of a packed quantised table, scaled;
`lora`    the low-rank adapters of the batch's requests, added beside a shared
          projection:  Y = Y0 + scale_a * B_a (A_a x);
`sample`  the next token of every request from its logits and a given random
          number: temperature, top-k, top-p, min-p.

Free pages are a ring of n_pages entries, `ring` = (first, count) of its free
ones.  A request with n_new < 0 has ended: its pages join the ring's end.

Packed tables (nb = K / 32 blocks, ns = K / 256 super-blocks a row):
    q8_0  rows * nb 32-byte codes (code + 128), then rows * nb f16 d; w = d q
    q4_0  rows * nb 16-byte nibbles in element order, then rows * nb f16 d; w = d (q - 8)
    q4_k  rows * ns 128 bytes of nibbles, then rows * ns records {f16 d, f16 dmin,
          12 bytes of 6-bit scales and minima}; w = d sc q - dmin m
    q6_k  rows * ns 128 bytes of low nibbles, rows * ns 16 words of top bits,
          rows * ns 16 int8 scales, rows * ns f16 d; w = d sc (q - 32)
"""

import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_BYTES = {"q8_0": 34 / 32, "q4_0": 18 / 32, "q4_k": 144 / 256, "q6_k": 210 / 256}  # of one weight


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few requests over a small vocabulary of odd size, each with its own settings: all latency
        dict(name="sample_3x1021_f16", op="sample", type="f16", n=3, vocab=1021, settings="mixed", pad=3),
        # one user's next token, nucleus sampling over the tied embedding's vocabulary
        dict(name="sample_1x262144_f32", op="sample", type="f32", n=1, vocab=262144, settings="nucleus", pad=0),
        # a serving batch of requests that each chose their own settings, rows of odd length
        dict(name="sample_56x65537_bf16", op="sample", type="bf16", n=56, vocab=65537, settings="mixed", pad=7),
        # the largest batch's logits
        dict(name="sample_160x262144_f32", op="sample", type="f32", n=160, vocab=262144, settings="mixed", pad=0),
        # one user's token through one adapter of the output projection
        dict(name="lora_1_f32", op="lora", type="bf16", act="f32", tokens=1, n_seq=1, adapters=4, rank=16, K=4096,
             rows=5376, bare=0.0),
        # a decode batch in which nearly every request has its own adapter
        dict(name="lora_64_f32", op="lora", type="bf16", act="f32", tokens=64, n_seq=64, adapters=48, rank=32, K=5376,
             rows=21504, bare=0.1),
        # prompts of odd lengths behind the fused norm, whose output is Q8_0
        dict(name="lora_7_prompts_q8", op="lora", type="f16", act="q8", tokens=1531, n_seq=7, adapters=3, rank=64, K=5376,
             rows=8192, bare=0.2),
        # a full prefill of a few requests beside the widest projection
        dict(name="lora_4096_q8", op="lora", type="bf16", act="q8", tokens=4096, n_seq=4, adapters=4, rank=16, K=5376,
             rows=21504, bare=0.0),
        # one token's row of the tied embedding
        dict(name="embed_1_q8_0", op="embed", format="q8_0", type="f32", tokens=1, K=5376, rows=262144),
        # a prefill's rows, tokens repeating as they do in text
        dict(name="embed_8192_q4_k", op="embed", format="q4_k", type="bf16", tokens=8192, K=5376, rows=262144),
        # a decode step of a serving batch: one new token each, some requests ended, some starting
        dict(name="plan_96", op="plan", n_seq=96, new=1, kv=4000, page=64, starting=0.03, ending=0.03),
        # admission of many prompts at once, into small pages
        dict(name="plan_1000_prompts", op="plan", n_seq=1000, new=120, kv=300, page=16, starting=0.5, ending=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "lora", "lora", "embed", "plan"])
    if op == "sample":
        vocab = _log_int(rng, 300, 262144)
        return {"op": op, "type": rng.choice(["f32", "f32", "bf16", "f16"]), "vocab": vocab, "pad": rng.randint(0, 9),
                "n": _log_int(rng, 1, min(256, 160 * 262144 // (vocab + 9))), "settings": rng.choice(["mixed", "nucleus", "open"])}
    if op == "lora":
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        tokens = _log_int(rng, 1, 4096)
        K, rows = 32 * _log_int(rng, 16, 168), 4 * _log_int(rng, 128, 5376)
        # bounded by the largest listed case's products and by 1 GB of adapters
        tokens = max(1, min(tokens, 4 * 4096 * 16 * 26880 // (rank * (K + rows))))
        return {"op": op, "type": rng.choice(["bf16", "f16"]), "act": rng.choice(["f32", "q8"]), "tokens": tokens,
                "n_seq": tokens if rng.random() < 0.5 and tokens <= 256 else _log_int(rng, 1, min(tokens, 32)),
                "adapters": max(1, min(_log_int(rng, 1, 64), (1 << 29) // (rank * (K + rows)))), "rank": rank, "K": K,
                "rows": rows, "bare": rng.choice([0.0, 0.2, 0.5])}
    if op == "embed":
        fmt = rng.choice(["q8_0", "q4_0", "q4_k", "q6_k"])
        K = 256 * _log_int(rng, 2, 21)
        return {"op": op, "format": fmt, "type": rng.choice(["f32", "bf16", "f16"]), "tokens": _log_int(rng, 1, 8192), "K": K,
                "rows": _log_int(rng, 1000, 262144)}
    n_seq = _log_int(rng, 1, 1000)
    return {"op": op, "n_seq": n_seq, "new": 1 if rng.random() < 0.5 else _log_int(rng, 2, max(2, min(4096, 120000 // n_seq))),
            "kv": _log_int(rng, 1, 8192), "page": rng.choice([16, 32, 64, 128]), "starting": round(rng.uniform(0.0, 0.5), 3),
            "ending": round(rng.uniform(0.0, 0.3), 3)}


def _spread(b, step):
    """Numbers spread evenly over [0, 1), the same for every run of a case."""
    return (b * step + 0.5) % 1.0


def _plan_lengths(case):
    """(new tokens, cached tokens) of every request; new = -1 for one that has ended."""
    got = []
    for b in range(case["n_seq"]):
        f, g, h = (_spread(b, s) for s in (0.6180339887498949, 0.7548776662466927, 0.5698402909980532))
        kv = 1 + int((case["kv"] - 1) * f)
        new = 1 + int((case["new"] - 1) * g)
        if h < case["ending"]:
            got.append((-1, kv))
        elif h > 1.0 - case["starting"]:
            got.append((1 + int(4 * case["new"] * f), 0))
        else:
            got.append((new, kv))
    return got


def _lora_rows(case):
    """(tokens, adapter) of every request; adapter -1 where it has none."""
    n, m = case["n_seq"], case["tokens"]
    weight = [0.3 + _spread(b, 0.6180339887498949) for b in range(n)]
    total, at, done = sum(weight), 0.0, 0
    got = []
    for b in range(n):
        at += weight[b]
        end = m if b == n - 1 else max(done, min(m, int(round(m * at / total)))) if n < m else b + 1
        bare = _spread(b, 0.7548776662466927) < case["bare"]
        got.append((end - done, -1 if bare else (b * 7 + b // 3) % case["adapters"]))
        done = end
    return got


def work(case):
    if case["op"] == "sample":
        n = case["n"] * case["vocab"]
        # every logit once; a difference, an exponential and a sum each
        return {"bytes": n * _SIZE[case["type"]] + 28 * case["n"], "flops": 4 * n}
    if case["op"] == "lora":
        rows = _lora_rows(case)
        m = sum(t for t, a in rows if a >= 0)
        used = len({a for t, a in rows if a >= 0 and t > 0})
        x = 4 if case["act"] == "f32" else 36 / 32
        r = case["rank"]
        return {"bytes": used * r * (case["K"] + case["rows"]) * 2 + m * case["K"] * x + 8 * case["tokens"] * case["rows"],
                "flops": 2 * m * r * (case["K"] + case["rows"])}
    if case["op"] == "embed":
        # every token's row written, every distinct row read: at most as many as there are tokens
        m, k = case["tokens"], case["K"]
        distinct = case["rows"] * (1.0 - (1.0 - 1.0 / case["rows"]) ** m) if m > 1 else 1
        return {"bytes": 4 * m + m * k * _SIZE[case["type"]] + min(distinct, m) * k * _BYTES[case["format"]], "flops": 2 * m * k}
    lens = _plan_lengths(case)
    page = case["page"]
    tokens = sum(max(0, n) for n, _ in lens)
    pages = sum(-(-kv // page) if n < 0 else -(-(kv + n) // page) - -(-kv // page) for n, kv in lens)
    return {"bytes": 16 * len(lens) + 16 * tokens + 8 * pages, "flops": 6 * tokens + 10 * len(lens)}


# ---------------------------------------------------------------- what a user has in hand

def _settings(case, g):
    """Every request's temperature, top-k, top-p and min-p."""
    n = case["n"]

    def pick(values):
        return torch.tensor(values, device="cuda")[torch.randint(len(values), (n,), generator=g, device="cuda")]

    if case["settings"] == "nucleus":
        return pick([0.7, 0.8, 1.0]).float(), pick([0]).int(), pick([0.9, 0.95]).float(), pick([0.0]).float()
    if case["settings"] == "open":
        return pick([0.8, 1.0, 1.2]).float(), pick([0]).int(), pick([1.0]).float(), pick([0.0, 0.0, 0.02]).float()
    return (pick([0.0, 0.3, 0.7, 0.8, 1.0, 1.0, 1.3]).float(), pick([0, 0, 0, 1, 20, 50, 200, 5000]).int(),
            pick([1.0, 0.5, 0.9, 0.95, 0.99]).float(), pick([0.0, 0.0, 0.02, 0.1]).float())


def _prepare_sample(case, g):
    n, vocab = case["n"], case["vocab"]
    # logits whose probabilities fall with the rank like a power between 1.2 and 2.5, as a language model's do
    x = torch.empty(n, vocab + case["pad"], device="cuda").exponential_(generator=g)
    x *= 1.2 + 1.3 * torch.rand(n, 1, generator=g, device="cuda")
    x -= 6.0
    # a fifth of the requests may only use some of the tokens
    only = torch.rand(n, 1, generator=g, device="cuda") < 0.2
    x.masked_fill_(only & (torch.rand(n, x.shape[1], generator=g, device="cuda") < 0.9), -math.inf)
    x = x.to(_TYPES[case["type"]])
    t, k, p, m = _settings(case, g)
    return {"logits": x[:, :vocab], "temperature": t, "top_k": k, "top_p": p, "min_p": m,
            "u": torch.rand(n, generator=g, device="cuda"), "token": torch.empty(n, dtype=torch.int32, device="cuda"),
            "prob": torch.empty(n, device="cuda")}


def _prepare_lora(case, g):
    m, k, rows, r, na = (case[x] for x in ("tokens", "K", "rows", "rank", "adapters"))
    typ = _TYPES[case["type"]]
    lens = _lora_rows(case)
    state = {"A": (torch.randn(na, r, k, generator=g, device="cuda") * k ** -0.5).to(typ),
             "B": (torch.randn(na, rows, r, generator=g, device="cuda") * 0.3).to(typ),
             "scale": 0.5 + torch.rand(na, generator=g, device="cuda"),
             "adapter": torch.tensor([a for _, a in lens], dtype=torch.int32, device="cuda"),
             "lens": lens,
             # which request every token belongs to, as the plan says it
             "sequence": torch.tensor([b for b, (t, _) in enumerate(lens) for _ in range(t)], dtype=torch.int32, device="cuda"),
             "Y0": torch.randn(m, rows, generator=g, device="cuda"), "Y": torch.empty(m, rows, device="cuda")}
    x = torch.randn(m, k, generator=g, device="cuda")
    if case["act"] == "q8":
        d = x.view(m, k // 32, 32).abs().amax(-1) / 127.0
        state["Xq"] = torch.round(x.view(m, k // 32, 32) / d[..., None]).to(torch.int8).view(m, k)
        state["dx"] = d
    else:
        state["X"] = x
    return state


def _prepare_embed(case, g):
    rows, k, m, fmt = case["rows"], case["K"], case["tokens"], case["format"]
    n = int(rows * k * _BYTES[fmt])
    table = torch.randint(-(1 << 62), 1 << 62, (-(-n // 8),), generator=g, device="cuda").view(torch.uint8)[:n]
    # the super-scales (f16) among the random codes: small positive numbers
    planes = _planes(table, fmt, rows, k)
    for x in (planes[-1][..., :4] if fmt == "q4_k" else planes[-1],):
        half = torch.rand(x.shape[:-1] + (x.shape[-1] // 2,), generator=g, device="cuda") * 0.01 + 0.001
        x.copy_(half.to(torch.float16).view(torch.uint8))
    # few tokens make up most of a text
    ids = (rows * torch.rand(m, generator=g, device="cuda") ** 3).to(torch.int32).clamp_(max=rows - 1)
    return {"table": table, "ids": ids, "scale": math.sqrt(k), "Y": torch.empty(m, k, dtype=_TYPES[case["type"]], device="cuda")}


def _prepare_plan(case, g):
    lens, page = _plan_lengths(case), case["page"]
    n = len(lens)
    have = [-(-kv // page) for _, kv in lens]
    want = [h if x < 0 else -(-(kv + x) // page) for h, (x, kv) in zip(have, lens)]
    max_pages = max(want) + 1
    n_pages = sum(have) + sum(w - h for w, h in zip(want, have)) + 17
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda")
    count = torch.tensor(have, device="cuda")
    table[torch.arange(max_pages, device="cuda")[None, :] < count[:, None]] = order[:sum(have)]
    first = int(torch.randint(n_pages, (1,), generator=g, device="cuda"))
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    left = n_pages - sum(have)
    free[(first + torch.arange(left, device="cuda")) % n_pages] = order[sum(have):]
    tokens = sum(max(0, x) for x, _ in lens)
    state = {"n_new": torch.tensor([x for x, _ in lens], dtype=torch.int32, device="cuda"),
             "kv_in": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
             "ring_in": torch.tensor([first, left], dtype=torch.int32, device="cuda"), "free": free, "table": table,
             "n_pages": n_pages, "max_pages": max_pages, "n_tokens": tokens + 5}  # a padded batch
    for name, size, typ in (("kv_len", n, torch.int32), ("q_start", n + 1, torch.int32), ("ring", 2, torch.int32),
                            ("slot", tokens + 5, torch.int64), ("position", tokens + 5, torch.int32),
                            ("sequence", tokens + 5, torch.int32)):
        state[name] = torch.empty(size, dtype=typ, device="cuda")
    return state


def prepare(case, seed):
    case = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"sample": _prepare_sample, "lora": _prepare_lora, "embed": _prepare_embed, "plan": _prepare_plan}[case["op"]](case, g)
    state["case"] = case
    if own and case["op"] in ("sample", "lora"):
        # the workspace that a program allocates once
        import block_quantized_matvec_gq_gb300 as gq
        size = (gq.gq_sample_workspace_bytes(case["vocab"], case["n"]) if case["op"] == "sample" else
                gq.gq_lora_workspace_bytes(case["rank"], case["K"], case["tokens"]))
        state["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return state


# ---------------------------------------------------------------- plain forms

def _plain_sample(s):
    """Largest logits first, equal ones by index; what is kept is always a beginning of that order."""
    l = s["logits"].float()
    n, vocab = l.shape
    l = torch.where(torch.isnan(l), -math.inf, l)
    l, order = torch.sort(l, dim=-1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    top = l[:, :1].double()
    w = torch.exp((l.double() - torch.where(torch.isfinite(top), top, 0.0)) / torch.where(t > 0, t, 1.0))
    k = s["top_k"].long()[:, None]
    at = torch.arange(vocab, device=l.device)[None, :]
    w *= (at < torch.where(k > 0, k, vocab)) & ((t > 0) | (at == 0))
    mass = torch.cumsum(w, -1)
    p = s["top_p"].double()[:, None]
    w *= (mass - w < p * mass[:, -1:]) | (p >= 1.0) | (at == 0)
    w *= w >= s["min_p"].double()[:, None] * w[:, :1]
    mass = torch.cumsum(w, -1)
    total = mass[:, -1:]
    j = (mass <= s["u"].double()[:, None] * total).sum(-1, keepdim=True).clamp(max=vocab - 1)
    some = total[:, 0] > 0
    token = torch.where(some, order.gather(1, j)[:, 0], -1).to(torch.int32)
    return {"token": token, "prob": torch.where(some, (w.gather(1, j) / total)[:, 0], 0.0).float()}


def _plain_lora(s):
    case = s["case"]
    a, b = s["A"].float(), s["B"].float()
    if case["act"] == "q8":
        m, k = s["Xq"].shape
        x = (s["Xq"].float().view(m, k // 32, 32) * s["dx"][..., None]).view(m, k)
    else:
        x = s["X"]
    # every token against every adapter at once, the others' parts masked away
    na, r = a.shape[:2]
    of = s["adapter"].long()[s["sequence"].long()]
    own_part = (of[:, None] == torch.arange(na, device=of.device)[None, :]) * s["scale"][None, :]
    v = (x @ a.flatten(0, 1).T).view(-1, na, r) * own_part[..., None]
    return s["Y0"] + v.flatten(1) @ b.transpose(1, 2).flatten(0, 1)


def _planes(table, fmt, rows, k):
    """Byte views of a packed table's planes, a row of the matrix each."""
    def cut(sizes):
        at, got = 0, []
        for n in sizes:
            got.append(table[at:at + rows * n].view(rows, n))
            at += rows * n
        return got

    nb, ns = k // 32, k // 256
    if fmt == "q4_k":
        q, rec = cut([128 * ns, 16 * ns])
        return q, rec.view(rows, ns, 16)
    return cut({"q8_0": [32 * nb, 2 * nb], "q4_0": [16 * nb, 2 * nb], "q6_k": [128 * ns, 64 * ns, 16 * ns, 2 * ns]}[fmt])


def _nibbles(x):
    return torch.stack((x & 15, x >> 4), -1).flatten(-2).float()


def _plain_embed(s):
    case = s["case"]
    fmt, k, m = case["format"], case["K"], case["tokens"]
    planes = [x[s["ids"].long()] for x in _planes(s["table"], fmt, case["rows"], k)]
    if fmt == "q8_0":
        w = (planes[0].float() - 128.0).view(m, k // 32, 32) * planes[1].view(torch.float16).float()[..., None]
    elif fmt == "q4_0":
        w = (_nibbles(planes[0]) - 8.0).view(m, k // 32, 32) * planes[1].view(torch.float16).float()[..., None]
    elif fmt == "q4_k":
        rec = planes[1]
        d = rec[..., :4].contiguous().view(torch.float16).float()  # d, dmin
        b = rec[..., 4:].int()
        lo, mid, hi = b[..., :4], b[..., 4:8], b[..., 8:]
        sc = torch.cat((lo & 63, (hi & 15) | (lo >> 6) << 4), -1).float()
        mn = torch.cat((mid & 63, (hi >> 4) | (mid >> 6) << 4), -1).float()
        q = _nibbles(planes[0]).view(m, k // 256, 8, 32)
        w = (d[..., :1] * sc)[..., None] * q - (d[..., 1:] * mn)[..., None]
    else:
        top = planes[1].contiguous().view(torch.int32)[..., None]
        bit = torch.tensor([4 * i + (0, 2, 16, 18)[a] for a in range(4) for i in range(4)], device=top.device)
        q = _nibbles(planes[0]).view(m, k // 16, 16) + ((top >> bit) & 3).view(m, k // 16, 16).float() * 16.0 - 32.0
        sc = planes[2].view(torch.int8).float() * planes[3].view(torch.float16).float().repeat_interleave(16, -1)
        w = q * sc[..., None]
    return (w.reshape(m, k) * s["scale"]).to(_TYPES[case["type"]])


def _plain_plan(s):
    page, n_pages, max_pages = s["case"]["page"], s["n_pages"], s["max_pages"]
    n_new, kv = s["n_new"].long(), s["kv_in"].long()
    first, count = s["ring_in"].long().unbind()
    ended = n_new < 0
    new = n_new.clamp(min=0)
    have, want = (kv + page - 1) // page, (kv + new + page - 1) // page
    need, back = torch.where(ended, 0, want - have), torch.where(ended, have, 0)
    need_at, back_at = torch.cumsum(need, 0) - need, torch.cumsum(back, 0) - back
    j = torch.arange(max_pages, device=kv.device)[None, :]
    taken = s["free"][(first + need_at[:, None] + j - have[:, None]) % n_pages]
    table = torch.where((j >= have[:, None]) & (j < want[:, None]) & ~ended[:, None], taken, s["table"])
    # pages that come back, behind the ring's last free one; the others' writes go to an entry that is cut off
    to = torch.where(ended[:, None] & (j < have[:, None]), (first + count + back_at[:, None] + j) % n_pages, n_pages)
    free = torch.cat((s["free"], s["free"][:1])).scatter(0, to.flatten(), s["table"].flatten())[:n_pages]
    ends = torch.cumsum(new, 0)
    q_start = torch.cat((ends.new_zeros(1), ends))
    t = torch.arange(s["n_tokens"], device=kv.device)
    real = t < ends[-1]
    seq = torch.searchsorted(ends, t, right=True).clamp(max=len(new) - 1)
    pos = kv[seq] + t - q_start[seq]
    slot = table[seq, (pos // page).clamp(max=max_pages - 1)].long() * page + pos % page
    return {"kv_len": torch.where(ended, 0, kv + new).int(), "q_start": q_start.int(), "table": table, "free": free,
            "ring": torch.stack(((first + need.sum()) % n_pages, count - need.sum() + back.sum())).int(),
            "slot": torch.where(real, slot, -1), "position": torch.where(real, pos, -1).int(),
            "sequence": torch.where(real, seq, -1).int()}


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return {"sample": _plain_sample, "lora": _plain_lora, "embed": _plain_embed, "plan": _plain_plan}[case["op"]](state)
    import block_quantized_matvec_gq_gb300 as gq

    s = state
    if case["op"] == "plan":
        gq.gq_kv_plan(s["n_new"], s["kv_in"], s["ring_in"], s["free"], s["table"], s["kv_len"], s["q_start"], s["ring"], s["slot"],
                      s["position"], s["sequence"], s["n_pages"], s["max_pages"], case["page"], case["n_seq"], s["n_tokens"])
        return {n: s[n] for n in ("kv_len", "q_start", "table", "free", "ring", "slot", "position", "sequence")}
    typ = {"f32": gq.GQ_TYPE_F32, "bf16": gq.GQ_TYPE_BF16, "f16": gq.GQ_TYPE_F16}[case["type"]]
    if case["op"] == "embed":
        fmt = {"q8_0": gq.GQ_FORMAT_Q8_0, "q4_0": gq.GQ_FORMAT_Q4_0, "q4_k": gq.GQ_FORMAT_Q4_K, "q6_k": gq.GQ_FORMAT_Q6_K}
        gq.gq_embed(fmt[case["format"]], s["table"], s["ids"], s["scale"], s["Y"], s["Y"].stride(0), typ, case["rows"], case["K"],
                    case["tokens"])
        return s["Y"]
    if case["op"] == "sample":
        gq.gq_sample(s["logits"], s["logits"].stride(0), typ, s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"],
                     s["token"], s["prob"], s["ws"], s["ws"].numel(), case["vocab"], case["n"])
        return {"token": s["token"], "prob": s["prob"]}
    sizes = (s["ws"], s["ws"].numel(), case["adapters"], case["rank"], case["rows"], case["K"], case["n_seq"], case["tokens"])
    lists = (s["scale"], s["adapter"], s["sequence"])
    y = (s["Y0"], s["Y0"].stride(0), s["Y"], s["Y"].stride(0))
    if case["act"] == "q8":
        gq.gq_lora_add_q8act(s["A"], s["B"], typ, *lists, s["Xq"], s["dx"], *y, *sizes)
    else:
        gq.gq_lora_add(s["A"], s["B"], typ, *lists, s["X"], s["X"].stride(0), *y, *sizes)
    return s["Y"]


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_sample(s):
    tokens, probs = [], []
    for row, t, k, p, m, u in zip(s["logits"].cpu().to(torch.float64).numpy(), *(s[x].cpu().double().numpy() for x in
                                  ("temperature", "top_k", "top_p", "min_p", "u"))):
        allowed = np.flatnonzero(row > -np.inf)
        if not allowed.size:
            tokens.append(-1)
            probs.append(0.0)
            continue
        ranked = allowed[np.argsort(-row[allowed], kind="stable")]
        if t <= 0:
            tokens.append(int(ranked[0]))
            probs.append(1.0)
            continue
        if k > 0:
            ranked = ranked[:int(k)]
        w = np.exp((row[ranked] - row[ranked[0]]) / t)
        n = len(w) if p >= 1 else 1 + int(np.searchsorted(np.cumsum(w), p * w.sum()))
        w = w[:n]
        w = w[:int(np.count_nonzero(w >= m))]
        at = min(int(np.searchsorted(np.cumsum(w), u * w.sum(), side="right")), len(w) - 1)
        tokens.append(int(ranked[at]))
        probs.append(float(w[at] / w.sum()))
    return {"token": np.array(tokens, dtype=np.int32), "prob": np.array(probs)}


def _exact_lora(s):
    x = s["X"].double() if "X" in s else s["Xq"].double() * s["dx"].double().repeat_interleave(32, -1)
    y = s["Y0"].double()
    of = torch.tensor([a for n, a in s["lens"] for _ in range(n)], device=y.device)
    for a in range(s["A"].shape[0]):
        rows = torch.nonzero(of == a)[:, 0]
        if len(rows):
            v = torch.einsum("tk,rk->tr", x[rows], s["A"][a].double())
            y[rows] += float(s["scale"][a]) * torch.einsum("tr,ir->ti", v, s["B"][a].double())
    return y


def _exact_embed(s):
    case = s["case"]
    fmt, k = case["format"], case["K"]
    ids, scale = s["ids"].cpu().numpy(), s["scale"]
    first, place = np.unique(ids, return_inverse=True)
    rows = [x[torch.from_numpy(first).long().cuda()].cpu().numpy() for x in _planes(s["table"], fmt, case["rows"], k)]
    e = np.arange(k)
    half = lambda x: x.copy().view(np.float16).astype(np.float64)  # noqa: E731
    if fmt == "q8_0":
        w = (rows[0].astype(np.float64) - 128) * half(rows[1])[:, e // 32]
    else:
        q = rows[0][:, e // 2] >> (4 * (e % 2)).astype(np.uint8) & 15
        if fmt == "q4_0":
            w = (q.astype(np.float64) - 8) * half(rows[1])[:, e // 32]
        elif fmt == "q4_k":
            rec, sub = rows[1], e // 32 % 8
            by = rec[:, e // 256, :]
            at = lambda i: np.take_along_axis(by, np.broadcast_to((4 + i)[None, :, None], by.shape[:2] + (1,)), -1)[..., 0]  # noqa: E731
            low = sub < 4
            sc = np.where(low, at(sub) & 63, (at(np.where(low, 0, sub + 4)) & 15) | (at(np.where(low, 0, sub - 4)) >> 6) << 4)
            mn = np.where(low, at(np.where(low, sub + 4, 0)) & 63, (at(np.where(low, 0, sub + 4)) >> 4) | (at(sub) >> 6) << 4)
            d = half(rec[..., :4].reshape(len(first), -1)).reshape(len(first), -1, 2)
            w = d[:, e // 256, 0] * sc * q - d[:, e // 256, 1] * mn
        else:
            word = rows[1].copy().view(np.uint32)[:, e // 16]
            place_of = np.array([0, 2, 16, 18])[e % 16 // 4] + 4 * (e % 4)
            q = q.astype(np.int64) + 16 * (word >> place_of.astype(np.uint32) & 3).astype(np.int64) - 32
            w = half(rows[3])[:, e // 256] * rows[2].view(np.int8)[:, e // 16] * q
    return (w * scale)[place.reshape(-1)]


def _exact_plan(s):
    page, n_pages = s["case"]["page"], s["n_pages"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    first, count = (int(x) for x in s["ring_in"].cpu())
    end = first + count
    kv_len, q_start, rows = [], [0], []
    for b, (n, kv) in enumerate(zip(s["n_new"].tolist(), s["kv_in"].tolist())):
        have = -(-kv // page)
        if n < 0:
            for j in range(have):
                free[end % n_pages] = table[b, j]
                end += 1
            n = kv = 0
        for j in range(have if kv else 0, -(-(kv + n) // page)):
            table[b, j] = free[first % n_pages]
            first += 1
        rows += [(int(table[b, x // page]) * page + x % page, x, b) for x in range(kv, kv + n)]
        kv_len.append(kv + n)
        q_start.append(q_start[-1] + n)
    rows += [(-1, -1, -1)] * (s["n_tokens"] - len(rows))
    slot, position, sequence = (np.array(x, dtype=np.int64) for x in zip(*rows))
    return {"kv_len": np.array(kv_len, np.int32), "q_start": np.array(q_start, np.int32), "table": table, "free": free,
            "ring": np.array([first % n_pages, end - first], np.int32), "slot": slot, "position": position.astype(np.int32),
            "sequence": sequence.astype(np.int32)}


def exact(case, seed):
    state = prepare(case, seed)
    return {"sample": _exact_sample, "lora": _exact_lora, "embed": _exact_embed, "plan": _exact_plan}[case["op"]](state)
