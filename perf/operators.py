"""Cases for the operators between a decode layer's qkv product and its output
product: block tables and slot maps (``slots``), rotary positions with the
write into the paged cache (``append``) and attention over that cache
(``attn``).  The head layout 32 query / 8 key heads of 128 is the 6144-row qkv
product of the 4096-wide decode layer this repository benchmarks.

``own = False`` computes every operator with elementary torch operations;
``own = True`` calls the library.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 64 requests: the map is built before every step, its latency is paid each time
        {"name": "slots_decode_64", "op": "slots", "requests": 64, "fresh": 1, "ragged": False, "cached": 8192, "page": 16,
         "pad": 0, "salt": 1},
        # a busy step: a thousand requests, chunks of new prompts among single tokens, padded to a captured size
        {"name": "slots_mixed_1024", "op": "slots", "requests": 1024, "fresh": 61, "ragged": True, "cached": 4096,
         "page": 32, "pad": 777, "salt": 2},
        # 8 columns, the most that one product call takes: f32 rows straight from the qkv product
        {"name": "append_decode_8", "op": "append", "tokens": 8, "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "axes": 1,
         "style": "halves", "src": "f32", "type": "bf16", "page": 16, "hnd": False, "far": 131072},
        # the chunk of a long prompt
        {"name": "append_chunk_8192", "op": "append", "tokens": 8192, "hq": 32, "hkv": 8, "dim": 128, "rot": 128, "axes": 1,
         "style": "halves", "src": "bf16", "type": "bf16", "page": 16, "hnd": False, "far": 1000000},
        # frames of a video: three axes, part of the head rotated, neighbours paired, a ragged token count
        {"name": "append_video_4097", "op": "append", "tokens": 4097, "hq": 16, "hkv": 16, "dim": 64, "rot": 48, "axes": 3,
         "style": "pairs", "src": "f16", "type": "f16", "page": 32, "hnd": True, "far": 2000},
        # one user's next token: latency
        {"name": "attn_token_1", "op": "attn", "requests": 1, "fresh": 1, "chunks": 0, "kv": 4099, "ragged": False, "hq": 32,
         "hkv": 8, "dim": 128, "type": "bf16", "page": 16, "hnd": False, "window": 0, "sinks": 0, "salt": 3},
        # a decode step of 64 requests of mixed age
        {"name": "attn_decode_64", "op": "attn", "requests": 64, "fresh": 1, "chunks": 0, "kv": 16384, "ragged": True,
         "hq": 32, "hkv": 8, "dim": 128, "type": "f16", "page": 16, "hnd": False, "window": 0, "sinks": 0, "salt": 4},
        # long chats under a sliding window with four first tokens kept
        {"name": "attn_window_16", "op": "attn", "requests": 16, "fresh": 1, "chunks": 0, "kv": 65536, "ragged": True,
         "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "page": 64, "hnd": False, "window": 4096, "sinks": 4, "salt": 5},
        # one token over a very long document
        {"name": "attn_long_131072", "op": "attn", "requests": 1, "fresh": 1, "chunks": 0, "kv": 131072, "ragged": False,
         "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "page": 32, "hnd": True, "window": 0, "sinks": 0, "salt": 6},
        # drafts of up to five tokens checked at once, wide heads, an odd group and page
        {"name": "attn_drafts_8", "op": "attn", "requests": 8, "fresh": 5, "chunks": 8, "kv": 2500, "ragged": True, "hq": 14,
         "hkv": 2, "dim": 256, "type": "bf16", "page": 24, "hnd": False, "window": 0, "sinks": 0, "salt": 7},
        # a chunk of a long prompt over what is cached of it: matrix work
        {"name": "attn_chunk_2048", "op": "attn", "requests": 1, "fresh": 2048, "chunks": 1, "kv": 8192, "ragged": False,
         "hq": 32, "hkv": 8, "dim": 128, "type": "bf16", "page": 16, "hnd": False, "window": 0, "sinks": 0, "salt": 8},
        # chunks of two prompts among single tokens, small heads, a window
        {"name": "attn_mixed_16", "op": "attn", "requests": 16, "fresh": 509, "chunks": 2, "kv": 4000, "ragged": True,
         "hq": 32, "hkv": 8, "dim": 64, "type": "f16", "page": 16, "hnd": False, "window": 1024, "sinks": 16, "salt": 9},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["slots", "append", "attn", "attn", "attn"])
    if op == "slots":
        return {"op": op, "requests": _spread(rng, 1, 1024), "fresh": _spread(rng, 1, 61), "ragged": rng.random() < 0.7,
                "cached": _spread(rng, 1, 8192), "page": rng.choice([1, 16, 24, 32, 64, 128]),
                "pad": rng.choice([0, 0, rng.randrange(1, 1000)]), "salt": rng.randrange(1 << 30)}
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8, 16])
        dim = rng.choice([64, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim - 32])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        return {"op": op, "tokens": _spread(rng, 1, max(1, min(8192, 8192 * 48 * 128 // ((hq + 2 * hkv) * dim)))),
                "hq": hq, "hkv": hkv, "dim": dim, "rot": rot, "axes": rng.choice([1, 1, 2, 3]),
                "style": rng.choice(["halves", "pairs"]), "src": rng.choice(["f32", "f16", "bf16"]),
                "type": rng.choice(["f16", "bf16"]), "page": rng.choice([1, 16, 24, 32, 64, 128]),
                "hnd": rng.random() < 0.5, "far": _spread(rng, 10, 1000000)}
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
            "page": rng.choice([1, 16, 16, 24, 32, 64, 128]), "hnd": rng.random() < 0.5,
            "window": rng.choice([0, 0, _spread(rng, 1, 8192)]), "sinks": rng.choice([0, 4, 16, 100]),
            "salt": rng.randrange(1 << 30)}
    while work(case)["flops"] > 2.4e11:
        case["kv"] = max(1, case["kv"] * 3 // 4)
        case["fresh"] = min(case["fresh"], case["kv"])
    return case


# ------------------------------------------------------------------ lengths (fixed by the case)

def _slots_lengths(case):
    r = random.Random(case["salt"])
    n = case["requests"]
    fresh = [r.randrange(0, 2 * case["fresh"]) if case["ragged"] else case["fresh"] for _ in range(n)]
    cached = [0 if r.random() < 0.2 else r.randrange(1, case["cached"] + 1) for _ in range(n)]  # 0: a new prompt
    fresh[0], cached[0] = max(1, fresh[0]), max(1, cached[0])
    return cached, fresh


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


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(case, pages, g, normal=True):
    """An empty or filled cache [pages, page, heads, dim]; "hnd" keeps a page's rows of one head together in memory."""
    shape = (pages, case["hkv"], case["page"], case["dim"]) if case["hnd"] else (pages, case["page"], case["hkv"], case["dim"])
    t = torch.randn(shape, generator=g, device="cuda", dtype=TYPES[case["type"]]) if normal else torch.zeros(
        shape, device="cuda", dtype=TYPES[case["type"]])
    return t.transpose(1, 2) if case["hnd"] else t


def prepare(case, seed):
    g = _generator(seed)
    page = case["page"]
    if case["op"] == "slots":
        cached, fresh = _slots_lengths(case)
        n, tokens = len(fresh), sum(fresh) + case["pad"]
        width = _pages(case["cached"] + 2 * case["fresh"], page)
        old = [_pages(c, page) for c in cached]
        need = sum(_pages(c + f, page) - o for c, f, o in zip(cached, fresh, old))
        ids = torch.randperm(sum(old) + need + 64, generator=g, device="cuda", dtype=torch.int32)
        table = torch.full((n, width), -1, device="cuda", dtype=torch.int32)
        inside = torch.arange(width, device="cuda")[None, :] < _ints(old)[:, None]
        table[inside] = ids[:sum(old)]
        empty = lambda k: torch.empty(k, device="cuda", dtype=torch.int32)  # noqa: E731
        return {"case": case, "cached": _ints(cached), "fresh": _ints(fresh), "free": ids[sum(old):].contiguous(),
                "table": table, "query_start": empty(n + 1), "kv_len": empty(n), "request": empty(tokens),
                "position": empty(tokens), "slot": empty(tokens), "used": empty(1), "tokens": tokens}
    if case["op"] == "append":
        t, hq, hkv, dim = case["tokens"], case["hq"], case["hkv"], case["dim"]
        rows = torch.randn((t, (hq + 2 * hkv) * dim), generator=g, device="cuda", dtype=TYPES[case["src"]])
        q, k, v = rows.split([hq * dim, hkv * dim, hkv * dim], dim=1)
        half = case["rot"] // 2
        inv = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        pages = _pages(t, page) + 3
        slot = torch.randperm(pages * page, generator=g, device="cuda")[:t].int()
        pos = torch.randint(0, case["far"], (case["axes"], t), generator=g, device="cuda", dtype=torch.int32)
        axis = (torch.arange(half, device="cuda") * case["axes"] // half).int()
        return {"case": case, "q": q.view(t, hq, dim), "k": k.view(t, hkv, dim), "v": v.view(t, hkv, dim), "inv_freq": inv,
                "slot": slot, "position": pos, "axis": axis, "k_cache": _cache(case, pages, g, False),
                "v_cache": _cache(case, pages, g, False),
                "q_out": torch.empty((t, hq, dim), device="cuda", dtype=TYPES[case["type"]])}
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
    dt = TYPES[case["type"]]
    # queries of a trained head point somewhere: a few keys stand out from the rest
    q = torch.randn((tokens, case["hq"], case["dim"]), generator=g, device="cuda", dtype=dt) * 1.5
    k_cache, v_cache = _cache(case, sum(used) + 2, g), _cache(case, sum(used) + 2, g)
    return {"case": case, "q": q, "k_cache": k_cache, "v_cache": v_cache, "table": table, "query_start": _ints(starts),
             "kv_len": _ints(kv), "scale": case["dim"] ** -0.5, "out": torch.empty_like(q), "most_new": max(fresh),
            "most_kv": max(kv),
            # scratch that a program keeps for its life, zero before its first use
            "scratch": torch.zeros(96 << 20, device="cuda", dtype=torch.uint8)}


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        from decode_gemv_elementwise_amd import paged

        s = state
        if op == "slots":
            paged.gemv_paged_slots(s["cached"], s["fresh"], s["free"], s["case"]["page"], s["table"], s["query_start"],
                                   s["kv_len"], s["request"], s["position"], s["slot"], s["used"])
            return {k: s[k] for k in ("table", "query_start", "kv_len", "request", "position", "slot", "used")}
        if op == "append":
            paged.gemv_paged_append(s["q"], s["k"], s["v"], s["position"], s["inv_freq"], s["slot"], s["q_out"],
                                    s["k_cache"], s["v_cache"], axis=s["axis"], style=s["case"]["style"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        paged.gemv_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["query_start"], s["kv_len"], s["scale"],
                              s["out"], s["scratch"], window=s["case"]["window"], sinks=s["case"]["sinks"])
        return s["out"]
    return {"slots": _plain_slots, "append": _plain_append, "attn": _plain_attn}[op](state)


def _plain_slots(s):
    page, tokens = s["case"]["page"], s["tokens"]
    cached, fresh = s["cached"].long(), s["fresh"].long()
    start = torch.cat([fresh.new_zeros(1), fresh.cumsum(0)])
    kv = cached + fresh
    old, new = (cached + page - 1) // page, (kv + page - 1) // page
    taken = (new - old).cumsum(0)
    j = torch.arange(s["table"].shape[1], device=cached.device)[None, :]
    at = ((taken - (new - old) - old)[:, None] + j).clamp(0, s["free"].numel() - 1)
    table = torch.where((j >= old[:, None]) & (j < new[:, None]), s["free"][at], s["table"])
    t = torch.arange(tokens, device=cached.device)
    there = t < start[-1]
    r = torch.searchsorted(start[1:], t, right=True).clamp(max=fresh.numel() - 1)
    pos = torch.where(there, cached[r] + t - start[r], 0)
    slot = torch.where(there, table[r, pos // page].long() * page + pos % page, -1)
    return {"table": table, "query_start": start.int(), "kv_len": kv.int(), "request": torch.where(there, r, -1).int(),
            "position": pos.int(), "slot": slot.int(), "used": taken[-1:].int()}


def _plain_turn(x, cos, sin, rot, style):
    x, rest = x[..., :rot].float(), x[..., rot:].float()
    if style == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:]
        x = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x, rest], -1)


def _plain_append(s):
    case = s["case"]
    angle = s["position"].double().t()[:, s["axis"].long()] * s["inv_freq"].double()  # [t, rot / 2]: far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    dt, page = TYPES[case["type"]], case["page"]
    q = _plain_turn(s["q"], cos, sin, case["rot"], case["style"]).to(dt)
    k = _plain_turn(s["k"], cos, sin, case["rot"], case["style"]).to(dt)
    at = (s["slot"].long() // page, s["slot"].long() % page)
    s["k_cache"][at] = k
    s["v_cache"][at] = s["v"].float().to(dt)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    case = s["case"]
    page, hkv, dim = case["page"], case["hkv"], case["dim"]
    group = case["hq"] // hkv
    most_new, most_kv = s["most_new"], s["most_kv"]
    start, kv_len = s["query_start"].long(), s["kv_len"].long()
    fresh = start[1:] - start[:-1]
    n = fresh.numel()
    dev = start.device
    j = torch.arange(most_kv, device=dev)
    id_ = s["table"][:, j // page].long().clamp(min=0)  # [n, kv]
    k = s["k_cache"][id_, (j % page)[None, :]].permute(0, 2, 3, 1).float().contiguous()  # [n, hkv, dim, kv]
    v = s["v_cache"][id_, (j % page)[None, :]].permute(0, 2, 1, 3).float().contiguous()  # [n, hkv, kv, dim]
    i = torch.arange(most_new, device=dev)
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
    t = torch.arange(s["q"].shape[0], device=dev)
    r = torch.searchsorted(start[1:], t, right=True)
    return o[r, t - start[r]].to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    if case["op"] == "slots":
        cached, fresh = _slots_lengths(case)
        page = case["page"]
        old, new = [_pages(c, page) for c in cached], [_pages(c + f, page) for c, f in zip(cached, fresh)]
        taken = sum(new) - sum(old)
        tails = sum(1 for c, f in zip(cached, fresh) if f and c % page)  # a last page that goes on being filled is looked up
        tokens = sum(fresh) + case["pad"]
        return {"bytes": 4 * (2 * len(fresh) + 2 * taken + tails + 2 * len(fresh) + 2 + 3 * tokens), "flops": 0}
    if case["op"] == "append":
        t, values = case["tokens"], (case["hq"] + 2 * case["hkv"]) * case["dim"]
        turned = t * (case["hq"] + case["hkv"]) * case["rot"] // 2
        return {"bytes": t * values * (_size(case["src"]) + 2) + 4 * t * (case["axes"] + 1) + 4 * case["rot"],
                "flops": 6 * turned}
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
    rows = sum(fresh) * case["hq"] * case["dim"]
    return {"bytes": 2 * (2 * keys * case["hkv"] * case["dim"] + 2 * rows), "flops": 4 * pairs * case["hq"] * case["dim"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"slots": _exact_slots, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)


def _exact_slots(s):
    page = s["case"]["page"]
    cached, fresh, free = s["cached"].tolist(), s["fresh"].tolist(), iter(s["free"].tolist())
    table = s["table"].tolist()
    start, kv, request, position, slot, used = [0], [], [], [], [], 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        for at in range(-(-c // page), -(-(c + f) // page)):
            table[r][at] = next(free)
            used += 1
        for p in range(c, c + f):
            request.append(r)
            position.append(p)
            slot.append(table[r][p // page] * page + p % page)
        start.append(start[-1] + f)
        kv.append(c + f)
    rest = s["tokens"] - len(slot)
    return {"table": _ints(table), "query_start": _ints(start), "kv_len": _ints(kv), "request": _ints(request + [-1] * rest),
            "position": _ints(position + [0] * rest), "slot": _ints(slot + [-1] * rest), "used": _ints([used])}


def _exact_append(s):
    case = s["case"]
    rot = case["rot"]
    half = rot // 2
    pos, inv, axis = s["position"].double(), s["inv_freq"].double(), s["axis"].long()
    first = torch.arange(half, device=pos.device) * (2 if case["style"] == "pairs" else 1)
    second = first + (1 if case["style"] == "pairs" else half)
    angle = torch.stack([pos[axis[i]] * inv[i] for i in range(half)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": turned(s["q"]), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    k, slot = turned(s["k"]), s["slot"].long()
    out["k_cache"][slot // case["page"], slot % case["page"]] = k
    out["v_cache"][slot // case["page"], slot % case["page"]] = s["v"].double()
    return out


def _exact_attn(s):
    case = s["case"]
    page, group = case["page"], case["hq"] // case["hkv"]
    start, kv = s["query_start"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for r, keys in enumerate(kv):
        n = start[r + 1] - start[r]
        ids = s["table"][r, :_pages(keys, page)].long()
        k, v = s["k_cache"][ids].flatten(0, 1)[:keys], s["v_cache"][ids].flatten(0, 1)[:keys]
        p = torch.arange(keys - n, keys, device=k.device)[:, None]
        j = torch.arange(keys, device=k.device)[None, :]
        seen = j <= p
        if case["window"]:
            seen = seen & ((p - j < case["window"]) | (j < case["sinks"]))
        for h in range(case["hq"]):
            logit = s["q"][start[r]:start[r + 1], h].double() @ k[:, h // group].double().t() * s["scale"]
            weight = torch.softmax(torch.where(seen, logit, -math.inf), -1)
            out[start[r]:start[r + 1], h] = weight @ v[:, h // group].double()
    return out
