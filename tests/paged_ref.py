"""Plain 64-bit references of the paged operators, on the CPU, key by key from
the definitions in include/gemv_paged.h, and the error bounds that the GPU
results are held to."""
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def slots(cached, fresh, free, page, table, tokens):
    """Lists in; the outputs of gemv_paged_slots as a dict of lists (the table a copy)."""
    table = [list(row) for row in table]
    start, kv, request, position, slot, used = [0], [], [], [], [], 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        c = max(c, 0)
        f = min(max(f, 0), tokens - start[-1])
        for j in range(-(-c // page), -(-(c + f) // page)):
            if j < len(table[r]):
                table[r][j] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + f):
            request.append(r)
            position.append(p)
            id_ = table[r][p // page] if p // page < len(table[r]) else -1
            s = id_ * page + p % page
            slot.append(s if id_ >= 0 and s < 2 ** 31 else -1)
        start.append(start[-1] + f)
        kv.append(c + f)
    rest = tokens - len(slot)
    return {"block_table": table, "query_start": start, "kv_len": kv, "token_request": request + [-1] * rest,
            "positions": position + [0] * rest, "slots": slot + [-1] * rest, "used": [used]}


def turned(x, positions, inv_freq, axis, pairs):
    """x [tokens, heads, dim] in 64 bits, its first 2 * len(inv_freq) values turned."""
    y = x.double().clone()
    half = inv_freq.numel()
    positions = positions.view(1, -1).double() if positions.dim() == 1 else positions.double()
    for i in range(half):
        ax = 0 if axis is None else int(axis[i])
        if not 0 <= ax < positions.shape[0]:
            continue
        lo, hi = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        angle = positions[ax] * inv_freq[i].double()
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        a, b = x[..., lo].double(), x[..., hi].double()
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def attn(q, k_cache, v_cache, table, query_start, kv_len, scale, window, sinks, out_dtype):
    """(result, bound, rows that belong to a request) in 64 bits on the CPU.

    The bound of one value counts: the weight's rounding to the cache's type
    (half a step u of the weights' mass A = sum w |v| / sum w; two pieces, u^2,
    for a float32 result), or binary16's smallest lifted step, 2^-39 of the
    largest weight, for each key; the float32 score's error d (its D products,
    the scaling, the exponent's own rounding), which moves the weights and their
    sum; float32 sums over the keys; and the result's rounding."""
    pu = HALF_STEP[k_cache.dtype]
    pu = pu * pu if out_dtype == torch.float32 else pu
    q, k_cache, v_cache = q.cpu().double(), k_cache.cpu().double(), v_cache.cpu().double()
    table, starts, lens = table.cpu().tolist(), query_start.cpu().tolist(), kv_len.cpu().tolist()
    pages, page, heads, dim = k_cache.shape
    tokens, q_heads, _ = q.shape
    group = q_heads // heads
    u = HALF_STEP[out_dtype]
    y, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    mine = torch.zeros(tokens, dtype=torch.bool)
    for r, kv in enumerate(lens):
        q0 = min(max(starts[r], 0), tokens)
        n = min(max(starts[r + 1], q0), tokens) - q0
        kv = max(kv, 0)
        mine[q0:q0 + n] = True
        js = [j for j in range(min(kv, len(table[r]) * page)) if 0 <= table[r][j // page] < pages]
        if not js or not n:
            continue
        j = torch.tensor(js)
        id_ = torch.tensor([table[r][x // page] for x in js])
        k, v = k_cache[id_, j % page], v_cache[id_, j % page]
        for i in range(n):
            p = kv - n + i
            see = j <= p
            if window:
                see &= (j > p - window) | (j < sinks)
            if not see.any():
                continue
            kk, vv = k[see].repeat_interleave(group, 1), v[see].repeat_interleave(group, 1)
            row = q[q0 + i]
            s = (kk * row).sum(-1) * scale  # [keys, q_heads]
            w = torch.exp(s - s.amax(0))
            w = torch.where(torch.isnan(s), s, w)
            total = w.sum(0)
            y[q0 + i] = (w[..., None] * vv).sum(0) / total[:, None]
            mass = (w[..., None] * vv.abs()).sum(0) / total[:, None]
            d = ((dim + 4) * 2.0 ** -24 * (kk * row).abs().sum(-1) * abs(scale) + 4 * 2.0 ** -24 * s.abs()).amax(0)
            n_keys = int(see.sum())
            rel = pu + 2 * d[:, None] + (n_keys / 8 + 128) * 2.0 ** -24
            small = n_keys * 2.0 ** -39 * vv.abs().amax(0) / total[:, None]
            bound[q0 + i] = mass * rel + small + u * y[q0 + i].abs() * 1.01
    return y, bound, mine
