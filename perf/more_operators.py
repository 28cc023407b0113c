"""Cases for the operators of a paged key/value cache held in 8 bits: rotary
positions with the quantising write and its reading back (``append``), tokens of
the cache in 16 or 32 bits (``read``), and attention over it (``attn``).  A block of
``block`` neighbouring tokens of a page has one scale for each head, a power of two
2^(byte - 127); codes are int8 or e4m3.  The head layout 32 query / 8 key heads of
128 is the 6144-row qkv product of the 4096-wide decode layer this repository
benchmarks.

``own = False`` computes every operator with elementary torch operations;
``own = True`` calls the library.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
MOST = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step of eight requests: one token each into blocks that are half full
        {"name": "append_decode_8", "op": "append", "requests": 8, "fresh": 1, "ragged": False, "cached": 1000, "pad": 0, "hq": 32,
         "hkv": 8, "dim": 128, "rot": 128, "style": "halves", "src": "f32", "type": "bf16", "code": "int8", "page": 16,
         "block": 16, "hnd": False, "salt": 1},
        # the chunk of a long prompt
        {"name": "append_chunk_8192", "op": "append", "requests": 1, "fresh": 8192, "ragged": False, "cached": 4000, "pad": 0,
         "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "style": "halves", "src": "bf16", "type": "bf16", "code": "e4m3", "page": 16,
         "block": 16, "hnd": False, "salt": 2},
        # many requests with a few tokens each, part of the head turned, neighbours paired, blocks shorter than a page
        {"name": "append_mixed_200", "op": "append", "requests": 200, "fresh": 9, "ragged": True, "cached": 300, "pad": 77,
         "hq": 16, "hkv": 16, "dim": 64, "rot": 48, "style": "pairs", "src": "f16", "type": "f16", "code": "int8", "page": 64,
         "block": 32, "hnd": True, "salt": 3},
        # a few tokens looked at, some without a place
        {"name": "read_few_100", "op": "read", "tokens": 100, "cached": 5000, "hkv": 8, "dim": 128, "out": "f32", "code": "e4m3",
         "page": 32, "block": 32, "hnd": False, "salt": 4},
        # a long prefix handed over to a cache of 16 bits
        {"name": "read_prefix_65536", "op": "read", "tokens": 65536, "cached": 70000, "hkv": 8, "dim": 128, "out": "bf16",
         "code": "int8", "page": 16, "block": 16, "hnd": True, "salt": 5},
        # one user's next token: latency
        {"name": "attn_token_1", "op": "attn", "requests": 1, "fresh": 1, "chunks": 0, "kv": 4099, "ragged": False, "hq": 32,
         "hkv": 8, "dim": 128, "type": "bf16", "code": "e4m3", "page": 16, "block": 16, "hnd": False, "window": 0, "sinks": 0,
         "salt": 6},
        # a decode step of 64 requests of mixed age
        {"name": "attn_decode_64", "op": "attn", "requests": 64, "fresh": 1, "chunks": 0, "kv": 16384, "ragged": True, "hq": 32,
         "hkv": 8, "dim": 128, "type": "f16", "code": "int8", "page": 16, "block": 16, "hnd": False, "window": 0, "sinks": 0,
         "salt": 7},
        # one token over a very long document
        {"name": "attn_long_131072", "op": "attn", "requests": 1, "fresh": 1, "chunks": 0, "kv": 131072, "ragged": False,
         "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "code": "e4m3", "page": 32, "block": 32, "hnd": True, "window": 0,
         "sinks": 0, "salt": 8},
        # long chats under a sliding window with four first tokens kept
        {"name": "attn_window_16", "op": "attn", "requests": 16, "fresh": 1, "chunks": 0, "kv": 65536, "ragged": True, "hq": 32,
         "hkv": 8, "dim": 128, "type": "bf16", "code": "int8", "page": 64, "block": 32, "hnd": False, "window": 4096, "sinks": 4,
         "salt": 9},
        # drafts of up to five tokens checked at once, wide heads, an odd group and page
        {"name": "attn_drafts_8", "op": "attn", "requests": 8, "fresh": 5, "chunks": 8, "kv": 2500, "ragged": True, "hq": 14,
         "hkv": 2, "dim": 256, "type": "bf16", "code": "e4m3", "page": 24, "block": 8, "hnd": False, "window": 0, "sinks": 0,
         "salt": 10},
        # a chunk of a long prompt over what is cached of it: matrix work
        {"name": "attn_chunk_2048", "op": "attn", "requests": 1, "fresh": 2048, "chunks": 1, "kv": 8192, "ragged": False,
         "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "code": "e4m3", "page": 16, "block": 16, "hnd": False, "window": 0,
         "sinks": 0, "salt": 11},
        # chunks of two prompts among single tokens, small heads, a window
        {"name": "attn_mixed_16", "op": "attn", "requests": 16, "fresh": 509, "chunks": 2, "kv": 4000, "ragged": True, "hq": 32,
         "hkv": 8, "dim": 64, "type": "f16", "code": "int8", "page": 16, "block": 16, "hnd": False, "window": 1024, "sinks": 16,
         "salt": 12},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def _paging(rng):
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    return {"page": page, "block": rng.choice([b for b in (4, 8, 16, 24, 32, 64) if page % b == 0]), "hnd": rng.random() < 0.5,
            "code": rng.choice(["int8", "e4m3"]), "salt": rng.randrange(1 << 30)}


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn"])
    if op == "append":
        hkv, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128, 256])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        requests = _spread(rng, 1, 256)
        most = max(1, 8192 * 48 * 128 // ((hq + 2 * hkv) * dim * requests))
        return {"op": op, "requests": requests, "fresh": _spread(rng, 1, min(most, 8192)) if rng.random() < 0.6 else 1,
                "ragged": rng.random() < 0.5, "cached": _spread(rng, 1, 1000), "pad": rng.choice([0, 0, rng.randrange(1, 100)]),
                "hq": hq, "hkv": hkv, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, dim - 32]),
                "style": rng.choice(["halves", "pairs"]), "src": rng.choice(["f32", "f16", "bf16"]),
                "type": rng.choice(["f16", "bf16"]), **_paging(rng)}
    if op == "read":
        hkv, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 128, 256])
        tokens = _spread(rng, 1, 65536 * 1024 // (16 * 256))
        return {"op": op, "tokens": tokens, "cached": tokens + rng.randrange(5000), "hkv": hkv, "dim": dim,
                "out": rng.choice(["f32", "f16", "bf16"]), **_paging(rng)}
    dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    kind = rng.choice(["tokens", "tokens", "drafts", "chunks", "mixed"])
    requests = _spread(rng, 1, 64 if kind in ("tokens", "drafts") else 16)
    fresh = {"tokens": 1, "drafts": rng.randrange(2, 9)}.get(kind) or _spread(rng, 9, 2048)
    chunks = {"tokens": 0, "mixed": rng.randrange(1, requests + 1)}.get(kind, requests)
    kv = _spread(rng, fresh, max(fresh, 32768))
    # what the plain form lays out at once (keys and scores, padded) stays under that of the largest listed cases
    while requests > 1 and (requests * kv * hkv * dim > (1 << 29) or requests * fresh * hq * kv > (1 << 29)):
        requests = (requests + 1) // 2
        chunks = min(chunks, requests)
    while fresh > 1 and fresh * hq * kv > (1 << 29):
        fresh = (fresh + 1) // 2
    case = {"op": op, "requests": requests, "fresh": fresh, "chunks": chunks, "kv": kv, "ragged": rng.random() < 0.7,
            "hq": hq, "hkv": hkv, "dim": dim, "type": rng.choice(["f16", "bf16"]),
            "window": rng.choice([0, 0, _spread(rng, 1, 8192)]), "sinks": rng.choice([0, 4, 16, 100]), **_paging(rng)}
    while work(case)["flops"] > 2.4e11:
        case["kv"] = max(1, case["kv"] * 3 // 4)
        case["fresh"] = min(case["fresh"], case["kv"])
    return case


# ------------------------------------------------------------------ lengths and places (fixed by the case)

def _pages(tokens, page):
    return -(-tokens // page)


def _append_lengths(case):
    """(cached tokens, new tokens) of every request."""
    r = random.Random(case["salt"])
    n = case["requests"]
    fresh = [r.randrange(0, 2 * case["fresh"]) if case["ragged"] else case["fresh"] for _ in range(n)]
    cached = [0 if r.random() < 0.2 else r.randrange(1, case["cached"] + 1) for _ in range(n)]  # 0: a new prompt
    fresh[0] = max(1, fresh[0])
    return cached, fresh


def _append_places(case):
    """(pages, slots of the new tokens, slots of all tokens in the blocks that get new ones, those blocks, each new token's
    block among them): the requests' pages lie scattered."""
    cached, fresh = _append_lengths(case)
    page, block = case["page"], case["block"]
    used = [_pages(c + f, page) for c, f in zip(cached, fresh)]
    ids = list(range(sum(used) + 3))
    random.Random(case["salt"] + 1).shuffle(ids)
    slots, there, blocks, row, at = [], [], [], [], 0
    for c, f, u in zip(cached, fresh, used):
        place = lambda p: ids[at + p // page] * page + p % page  # noqa: E731
        for p in range(c, c + f):
            if p == c or p % block == 0:
                blocks.append(place(p) // block)
            slots.append(place(p))
            row.append(len(blocks) - 1)
        if f:
            there += [place(p) for p in range(c // block * block, c + f)]
        at += u
    return len(ids), slots, there, blocks, row


def _attn_lengths(case):
    """(new tokens, key count) of every request; the chunks' places are drawn too."""
    r = random.Random(case["salt"])
    n = case["requests"]
    fresh = [1] * n
    for i in r.sample(range(n), case["chunks"]):
        fresh[i] = r.randrange(max(1, case["fresh"] // 2), case["fresh"] + 1) if case["ragged"] else case["fresh"]
    kv = [r.randrange(f, max(f, case["kv"]) + 1) if case["ragged"] else max(f, case["kv"]) for f in fresh]
    if case["ragged"]:
        kv[r.randrange(n)] = max(case["kv"], case["fresh"])
    return fresh, kv


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _byte_of(amax, code):
    """The scale's byte of a block whose largest size is amax: the least from 1 up with amax <= MOST 2^(byte - 127)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 127 = 0.9921875 * 2^7, 448 = 0.875 * 2^9
    e = e - torch.where(m <= 0.9921875, 7, 6) if code == "int8" else e - torch.where(m <= 0.875, 9, 8)
    return torch.where(amax > 0, e + 127, 1).clamp(1, 254)


def _code_of(x, code):
    """Floats within the codes' range rounded to them, ties to even."""
    return torch.round(x).to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _power(e):
    """2^e in float32, e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _filled(case, pages, g, keys):
    """Codes [pages, page, heads, dim] of random values and their scales [pages, page / block, heads].  Some channels of keys
    are larger than the rest, and tokens differ in size.  "hnd" keeps a page's rows of one head together in memory."""
    page, block, hkv, dim = case["page"], case["block"], case["hkv"], case["dim"]
    codes = torch.empty((pages, hkv, page, dim) if case["hnd"] else (pages, page, hkv, dim), dtype=CODES[case["code"]], device="cuda")
    codes = codes.transpose(1, 2) if case["hnd"] else codes
    scales = torch.empty((pages, page // block, hkv), dtype=torch.uint8, device="cuda")
    gain = torch.where(torch.rand((hkv, dim), generator=g, device="cuda") < 0.03, 4.0 if keys else 1.0, 1.0)
    some = max(1, (1 << 27) // (page * hkv * dim))
    for p in range(0, pages, some):
        n = min(some, pages - p)
        x = torch.randn((n, page, hkv, dim), generator=g, device="cuda") * gain
        x *= torch.rand((n, page, 1, 1), generator=g, device="cuda") + 0.5
        x = x.view(n, page // block, block, hkv, dim)
        byte = _byte_of(x.abs().amax((2, 4)), case["code"])
        scales[p:p + n] = byte.to(torch.uint8)
        codes[p:p + n] = _code_of(x * _power(127 - byte)[:, :, None, :, None], case["code"]).view(n, page, hkv, dim)
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    page, hkv, dim = case["page"], case["hkv"], case["dim"]
    if case["op"] == "append":
        pages, slots, there, blocks, row = _append_places(case)
        t, hq = len(slots) + case["pad"], case["hq"]
        rows = torch.randn((t, (hq + 2 * hkv) * dim), generator=g, device="cuda", dtype=TYPES[case["src"]])
        q, k, v = rows.split([hq * dim, hkv * dim, hkv * dim], dim=1)
        half = case["rot"] // 2
        inv = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        kc, ks = _filled(case, pages, g, True)
        vc, vs = _filled(case, pages, g, False)
        back = lambda: torch.empty((len(there), hkv, dim), dtype=TYPES[case["type"]], device="cuda")  # noqa: E731
        return {"case": case, "q": q.view(t, hq, dim), "k": k.view(t, hkv, dim), "v": v.view(t, hkv, dim), "inv_freq": inv,
                "slot": _ints(slots + [-1] * case["pad"]), "position": torch.randint(0, 131072, (t,), generator=g, device="cuda", dtype=torch.int32),
                "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "there": _ints(there), "blocks": _ints(blocks),
                "row": _ints(row), "q_out": torch.empty((t, hq, dim), device="cuda", dtype=TYPES[case["type"]]), "k_back": back(),
                "v_back": back()}
    if case["op"] == "read":
        kc, ks = _filled(case, _pages(case["cached"], page), g, True)
        vc, vs = _filled(case, _pages(case["cached"], page), g, False)
        r = random.Random(case["salt"])
        runs = [i for i in range(_pages(case["cached"], page))]
        r.shuffle(runs)  # the pages of a sequence, one after the other
        slot = [p * page + i for p in runs for i in range(page)][:case["tokens"]]
        for i in r.sample(range(len(slot)), len(slot) // 50):  # places that hold no token
            slot[i] = -1
        out = lambda: torch.empty((len(slot), hkv, dim), dtype=TYPES[case["out"]], device="cuda")  # noqa: E731
        return {"case": case, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "slot": _ints(slot), "k_back": out(),
                "v_back": out()}
    fresh, kv = _attn_lengths(case)
    n, tokens = len(fresh), sum(fresh)
    used = [_pages(k, page) for k in kv]
    ids = torch.randperm(sum(used) + 2, generator=g, device="cuda", dtype=torch.int32)
    width = max(used)
    table = torch.full((n, width), -1, device="cuda", dtype=torch.int32)
    inside = torch.arange(width, device="cuda")[None, :] < _ints(used)[:, None]
    table[inside] = ids[:sum(used)]
    starts = [0]
    for f in fresh:
        starts.append(starts[-1] + f)
    q = torch.randn((tokens, case["hq"], dim), generator=g, device="cuda", dtype=TYPES[case["type"]])
    kc, ks = _filled(case, sum(used) + 2, g, True)
    vc, vs = _filled(case, sum(used) + 2, g, False)
    return {"case": case, "q": q, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "table": table,
            "query_start": _ints(starts), "kv_len": _ints(kv), "scale": dim ** -0.5, "out": torch.empty_like(q),
            "most_new": max(fresh), "most_kv": max(kv),
            # scratch that a program keeps for its life, zero before its first use
            "scratch": torch.zeros(96 << 20, device="cuda", dtype=torch.uint8)}


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        from decode_gemv_elementwise_amd import paged8

        s = state
        cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if op == "append":
            paged8.gemv_paged8_append(s["q"], s["k"], s["v"], s["position"], s["inv_freq"], s["slot"], s["q_out"], *cache,
                                      style=s["case"]["style"])
            paged8.gemv_paged8_read(*cache, s["there"], s["k_back"], s["v_back"])
            return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}
        if op == "read":
            paged8.gemv_paged8_read(*cache, s["slot"], s["k_back"], s["v_back"])
            return {"k": s["k_back"], "v": s["v_back"]}
        paged8.gemv_paged8_attn(s["q"], *cache, s["table"], s["query_start"], s["kv_len"], s["scale"], s["out"], s["scratch"],
                                window=s["case"]["window"], sinks=s["case"]["sinks"])
        return s["out"]
    return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn}[op](state)


def _plain_turn(x, cos, sin, rot, style):
    x, rest = x[..., :rot].float(), x[..., rot:].float()
    if style == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:]
        x = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x, rest], -1)


def _plain_write(s, x, codes, scales):
    """x [tokens, heads, dim] into the blocks of this call (each listed once), those rescaled first where they have to be."""
    case = s["case"]
    page, block, hkv, dim = case["page"], case["block"], case["hkv"], case["dim"]
    blocks, row = s["blocks"].long(), s["row"].long()
    id_, part = blocks * block // page, blocks * block % page // block
    place = s["slot"].long()[:row.numel()] % block
    x = x[:row.numel()]
    amax = torch.zeros((blocks.numel(), hkv), device=x.device).index_reduce_(0, row, x.abs().amax(-1), "amax")
    begun = torch.zeros(blocks.numel(), device=x.device).index_reduce_(0, row, (place == 0).float(), "amax") > 0
    old = scales[id_, part].int()
    byte = _byte_of(amax, case["code"])
    byte = torch.where(begun[:, None], byte, torch.maximum(byte, old))
    at = part[:, None] * block + torch.arange(block, device=x.device)
    held = codes[id_[:, None], at].float() * _power((old - byte).clamp(min=-126))[:, None, :, None]
    held = torch.where(begun[:, None, None, None], 0.0, held)  # whatever lies there is no token's
    held[row, place] = x * _power(127 - byte)[row][..., None]
    codes[id_[:, None], at] = _code_of(held, case["code"])
    scales[id_, part] = byte.to(torch.uint8)


def _plain_values(codes, scales, slot, page, block, dtype):
    """The values of places of the cache, 0 where there is none."""
    at = slot.long().clamp(min=0)
    id_, place = at // page, at % page
    x = codes[id_, place].float() * _power(scales[id_, place // block].int() - 127)[..., None]
    return torch.where(slot[:, None, None] >= 0, x, 0.0).to(dtype)


def _plain_append(s):
    case = s["case"]
    angle = s["position"].double()[:, None] * s["inv_freq"].double()  # [t, rot / 2]: far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    dt = TYPES[case["type"]]
    q = _plain_turn(s["q"], cos, sin, case["rot"], case["style"]).to(dt)
    _plain_write(s, _plain_turn(s["k"], cos, sin, case["rot"], case["style"]), s["k_cache"], s["k_scale"])
    _plain_write(s, s["v"].float(), s["v_cache"], s["v_scale"])
    return {"q": q, "k": _plain_values(s["k_cache"], s["k_scale"], s["there"], case["page"], case["block"], dt),
            "v": _plain_values(s["v_cache"], s["v_scale"], s["there"], case["page"], case["block"], dt)}


def _plain_read(s):
    case = s["case"]
    return {x: _plain_values(s[x + "_cache"], s[x + "_scale"], s["slot"], case["page"], case["block"], TYPES[case["out"]])
            for x in "kv"}


def _plain_attn(s):
    case = s["case"]
    page, block, hkv, dim = case["page"], case["block"], case["hkv"], case["dim"]
    group = case["hq"] // hkv
    most_new, most_kv = s["most_new"], s["most_kv"]
    start, kv_len = s["query_start"].long(), s["kv_len"].long()
    fresh = start[1:] - start[:-1]
    n = fresh.numel()
    j = torch.arange(most_kv, device=start.device)
    id_ = s["table"][:, j // page].long().clamp(min=0)  # [n, kv]
    k = s["k_cache"][id_, (j % page)[None, :]].float()  # [n, kv, hkv, dim]
    k *= _power(s["k_scale"][id_, (j % page // block)[None, :]].int() - 127)[..., None]
    k = k.permute(0, 2, 3, 1).contiguous()
    v = s["v_cache"][id_, (j % page)[None, :]].float()
    v *= _power(s["v_scale"][id_, (j % page // block)[None, :]].int() - 127)[..., None]
    v = v.permute(0, 2, 1, 3).contiguous()
    i = torch.arange(most_new, device=start.device)
    token = (start[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)  # [n, new]
    q = s["q"][token].float().reshape(n, most_new, hkv, group, dim).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, hkv, group * most_new, dim)
    score = torch.matmul(q, k).mul_(s["scale"]).view(n, hkv, group, most_new, most_kv)
    p = (kv_len - fresh)[:, None] + i[None, :]  # [n, new]
    seen = (j <= p[..., None]) & (j < kv_len[:, None, None])
    if case["window"]:
        seen &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(n, hkv, group * most_new, most_kv), v).view(n, hkv, group, most_new, dim) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most_new, case["hq"], dim)
    t = torch.arange(s["q"].shape[0], device=start.device)
    r = torch.searchsorted(start[1:], t, right=True)
    return o[r, t - start[r]].to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    hkv, dim, block = case["hkv"], case["dim"], case["block"]
    if case["op"] == "append":
        _, slots, there, blocks, _ = _append_places(case)
        t, hq = len(slots) + case["pad"], case["hq"]
        read = t * hq + 2 * len(slots) * hkv  # heads of q, and of k and v with a place
        turned = (t * hq + len(slots) * hkv) * case["rot"] // 2
        return {"bytes": dim * (read * _size(case["src"]) + t * hq * 2 + 2 * len(slots) * hkv) + 2 * len(blocks) * hkv * 2 + 8 * t
                + 2 * case["rot"] + 2 * len(there) * hkv * dim * 3 + 4 * len(there), "flops": 6 * turned}
    if case["op"] == "read":
        tokens = case["tokens"]
        return {"bytes": 2 * tokens * hkv * (dim * (1 + _size(case["out"]))) + 2 * tokens * hkv // block + 4 * tokens, "flops": 0}
    fresh, kv = _attn_lengths(case)
    window, sinks = case["window"], case["sinks"]
    keys = pairs = 0
    for f, k in zip(fresh, kv):
        if window:
            low = max(0, k - f - window + 1)  # the first key that the first new token's window reaches
            keys += k - low + min(sinks, low)
            for p in range(k - f, k):
                edge = max(0, p - window + 1)
                pairs += p + 1 - edge + min(sinks, edge)
        else:
            keys += k
            pairs += f * (k - f) + f * (f + 1) // 2
    rows = sum(fresh) * case["hq"] * dim
    return {"bytes": 2 * keys * hkv * dim + 2 * keys * hkv // block + 4 * rows, "flops": 4 * pairs * case["hq"] * dim}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)


def _exact_values(s, name):
    """All values of the cache, [pages, page, heads, dim]."""
    byte = s[name + "_scale"].repeat_interleave(s["case"]["block"], 1).double()
    return s[name + "_cache"].float().double() * torch.exp2(byte - 127)[..., None]


def _exact_round(x, code):
    """x rounded to the codes' numbers: whole ones, or 4 significant bits down to steps of 2^-9."""
    if code == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    case = s["case"]
    rot, code, block = case["rot"], case["code"], case["block"]
    half = rot // 2
    first = torch.arange(half, device="cuda") * (2 if case["style"] == "pairs" else 1)
    second = first + (1 if case["style"] == "pairs" else half)
    angle = s["position"].double()[:, None] * s["inv_freq"].double()[None, :]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    slots = s["slot"].tolist()
    order = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            order.setdefault(slot // block, []).append(t)
    out = {"q": turned(s["q"])}
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        x = x.cpu()
        codes = s[name + "_cache"].float().double().cpu().flatten(0, 1)
        bytes_ = s[name + "_scale"].double().cpu().flatten(0, 1)
        for b, tokens in order.items():
            amax = x[tokens].abs().amax((0, 2))
            new = torch.ceil(torch.log2(amax / MOST[code])) + 127
            new = new + (amax > MOST[code] * torch.exp2(new - 127)) - (amax <= MOST[code] * torch.exp2(new - 128)).double()
            if not any(slots[t] % block == 0 for t in tokens):
                new = torch.maximum(new, bytes_[b])
            part = codes[b * block:(b + 1) * block]
            part[:] = _exact_round(part * torch.exp2(bytes_[b] - new)[:, None], code)
            for t in tokens:
                codes[slots[t]] = _exact_round(x[t] * torch.exp2(127 - new)[:, None], code)
            bytes_[b] = new
        there = s["there"].long().cpu()
        out[name] = codes[there] * torch.exp2(bytes_[there // block] - 127)[..., None]
    return out


def _exact_read(s):
    slot = s["slot"].long()
    return {name: _exact_values(s, name).flatten(0, 1)[slot.clamp(min=0)] * (slot >= 0)[:, None, None] for name in "kv"}


def _exact_attn(s):
    case = s["case"]
    page, block, group = case["page"], case["block"], case["hq"] // case["hkv"]
    start, kv = s["query_start"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for r, keys in enumerate(kv):
        n = start[r + 1] - start[r]
        ids = s["table"][r, :_pages(keys, page)].long()
        kc, vc = s["k_cache"][ids], s["v_cache"][ids]
        ks, vs = (s[x][ids].repeat_interleave(block, 1).flatten(0, 1)[:keys].double() for x in ("k_scale", "v_scale"))
        p = torch.arange(keys - n, keys, device=out.device)[:, None]
        j = torch.arange(keys, device=out.device)[None, :]
        seen = j <= p
        if case["window"]:
            seen = seen & ((p - j < case["window"]) | (j < case["sinks"]))
        for h in range(case["hq"]):
            g = h // group
            k = kc[:, :, g].float().flatten(0, 1)[:keys].double() * torch.exp2(ks[:, g] - 127)[:, None]
            v = vc[:, :, g].float().flatten(0, 1)[:keys].double() * torch.exp2(vs[:, g] - 127)[:, None]
            logit = s["q"][start[r]:start[r + 1], h].double() @ k.t() * s["scale"]
            out[start[r]:start[r + 1], h] = torch.softmax(torch.where(seen, logit, -math.inf), -1) @ v
    return out
