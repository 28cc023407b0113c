"""The operators over a paged cache in 8 bits on the GPU against the 64-bit references
of paged8_ref: lengths, head layouts, types, strides, pages, blocks and masks where they
can go wrong, and what they promise about buffers, streams and graphs."""
import random

import pytest
import torch

import paged8_ref as ref
import paged_ref
from decode_gemv_elementwise_amd import paged, paged8

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = torch.int32
KINDS = [("int8", "f16"), ("int8", "bf16"), ("e4m3", "f16"), ("e4m3", "bf16")]


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=I32, device=device)


def random_codes(shape, code, g):
    """Codes that fill their range, zeros and the largest among them."""
    x = torch.randn(shape, generator=g, device="cuda") * ref.MOST[code] / 4
    x = x.clamp(-ref.MOST[code], ref.MOST[code])
    return x.round().to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


# ------------------------------------------------------------------ reading

@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("out", DTYPES)
def test_read_every_code_and_scale(code, out):
    """All 256 codes under scales from the least to the largest and NaN: exactly the value, rounded once."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.int8 if code == "int8" else torch.float8_e4m3fn)
    codes = codes.view(1, 1, 1, 256).expand(256, 1, 1, 256).contiguous().view(256, 1, 1, 256)
    byte = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1, 1)
    got = torch.full((256, 1, 256), 7.0, dtype=DTYPES[out], device="cuda")
    v = torch.full_like(got, 7.0)
    paged8.gemv_paged8_read(codes, codes.clone(), byte, byte.clone(), ints(list(range(256))), got, v)
    assert torch.equal(torch.nan_to_num(got.float(), 3.0), torch.nan_to_num(v.float(), 3.0))
    want = ref.values(codes, byte)[:, 0].to(torch.float64)
    got = got.cpu()
    same = (got == want.to(DTYPES[out])) | (torch.isnan(got) & torch.isnan(want))
    tiny = want.abs() < 2.0 ** -117  # may be taken as 0
    assert (same | (tiny & (got.double().abs() <= 2.0 ** -117))).all(), (~same & ~tiny).nonzero()[:5]


@pytest.mark.parametrize("tokens,heads,dim,page,block,hnd", [
    (1, 1, 16, 1, 1, False), (0, 2, 64, 16, 16, False), (7, 3, 48, 24, 8, True), (33, 8, 128, 16, 16, False), (100, 2, 512, 5, 1, True),
    (1000, 4, 256, 64, 32, False), (5000, 8, 128, 16, 4, True)])
@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("out", DTYPES)
def test_read_places(tokens, heads, dim, page, block, hnd, code, out):
    """Any places, some outside the cache (zeros); rows apart; what lies between rows stays as it is."""
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    pages = max(2, tokens // page // 2)
    shape = (pages, heads, page, dim) if hnd else (pages, page, heads, dim)
    k, v = random_codes(shape, code, g), random_codes(shape, code, g)
    if hnd:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks, vs = (torch.randint(90, 150, (pages, heads, page // block), generator=g, device="cuda", dtype=torch.int32).byte().transpose(1, 2)
              for _ in "kv")
    slots = torch.randint(-3, pages * page + 3, (tokens,), generator=g, device="cuda", dtype=I32)
    if tokens > 3:
        slots[1], slots[2] = -2 ** 31, 2 ** 31 - 1
    wide = torch.full((2, tokens, heads * dim + 8), 7.0, dtype=DTYPES[out], device="cuda")
    outs = [w[:, :heads * dim].unflatten(1, (heads, dim)) for w in wide]
    paged8.gemv_paged8_read(k, v, ks, vs, slots, *outs)
    for codes, byte, got in ((k, ks, outs[0]), (v, vs, outs[1])):
        want = ref.values(codes, byte).flatten(0, 1)
        s = slots.cpu().long()
        there = (s >= 0) & (s < pages * page)
        want = torch.where(there[:, None, None], want[s.clamp(0, pages * page - 1)], 0.0).to(DTYPES[out])
        assert got.cpu().equal(want)
    assert (wide[:, :, heads * dim:] == 7).all()
    first, before = (o.clone() for o in outs)
    outs[0].fill_(7.0)
    paged8.gemv_paged8_read(k, v, ks, vs, slots, k_out=None, v_out=outs[1])
    assert (outs[0] == 7).all() and outs[1].equal(before)
    again = torch.empty_like(before.contiguous())
    paged8.gemv_paged8_read(k, v, ks, vs, slots, k_out=again)
    assert (outs[0] == 7).all() and again.equal(first)


# ------------------------------------------------------------------ writing

class Cache:
    """A cache that holds something everywhere, in either order of memory, scales with heads or blocks innermost."""

    def __init__(self, code, pages, page, block, heads, dim, hnd=False, seed=0, byte=(110, 125)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (pages, heads, page, dim) if hnd else (pages, page, heads, dim)
        self.k, self.v = random_codes(shape, code, g), random_codes(shape, code, g)
        if hnd:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        s = (pages, heads, page // block) if hnd else (pages, page // block, heads)
        self.ks, self.vs = (torch.randint(*byte, s, generator=g, device="cuda", dtype=torch.int32).byte() for _ in "kv")
        if hnd:
            self.ks, self.vs = self.ks.transpose(1, 2), self.vs.transpose(1, 2)
        self.code, self.page, self.block = code, page, block

    @property
    def all(self):
        return self.k, self.v, self.ks, self.vs

    def copy(self):
        return [t.cpu().clone() for t in self.all]


def held(c, before, slots, x, which, slack):
    """What a write of x [tokens, heads, dim] (64 bits) left in the cache's k or v: each scale by its definition, each new
    code within half its step of x (and `slack` for x's own computation), each old one rescaled, the rest as it was."""
    codes, bytes_ = (c.k, c.ks) if which == "k" else (c.v, c.vs)
    old, old_bytes = (before[0], before[2]) if which == "k" else (before[1], before[3])
    code, block = c.code, c.block
    heads = codes.shape[2]
    n = codes.shape[0] * codes.shape[1]
    got = codes.cpu().float().double().reshape(n // block, block, heads, -1)
    old = old.float().double().reshape(got.shape)
    gb, ob = (t.cpu().reshape(n // block, heads).long() for t in (bytes_, old_bytes))
    runs = {}
    for t, s in enumerate(slots):
        if 0 <= s < n:
            runs.setdefault(s // block, {})[s % block] = t
    touched = torch.zeros(n // block, dtype=torch.bool)
    rel, least = ref.HALF[code]
    for b, tokens in runs.items():
        touched[b] = True
        places = sorted(tokens)
        new = x[[tokens[p] for p in places]]  # [n, heads, dim]
        others = [p for p in range(block) if p not in tokens]
        for h in range(heads):
            amax = float(new[:, h].abs().max()) if torch.isfinite(new[:, h]).all() else float("nan")
            allowed = {ref.byte_for(a, code) for a in (amax, amax * (1 - 2.0 ** -20) - slack, amax * (1 + 2.0 ** -20) + slack)} \
                if slack else {ref.byte_for(amax, code)}
            if 0 not in tokens:
                allowed = {max(a, int(ob[b, h])) for a in allowed}
            byte = int(gb[b, h])
            assert byte in allowed, f"{which} block {b} head {h}: byte {byte}, expected {allowed}"
            if byte == 255:
                continue
            s = 2.0 ** (byte - 127)
            err = (got[b, places, h] * s - new[:, h]).abs()
            tol = torch.maximum(rel * new[:, h].abs(), torch.tensor(least * s)) * (1 + 2.0 ** -30) + slack
            assert (err <= tol).all(), f"{which} block {b} head {h}: off by {float((err - tol).max()):.3e} beyond half a step"
            if 0 not in tokens and others:
                want = ref.rounded(old[b, others, h] * 2.0 ** (int(ob[b, h]) - byte), code)
                assert got[b, others, h].equal(want), f"{which} block {b} head {h}: old codes"
    assert got[~touched].equal(old[~touched]) and gb[~touched].equal(ob[~touched]), f"{which}: another block was written"


def run_append(c, src, dtype, slots, hq, rot, axes=1, style="halves", shift=0, far=100000, seed=0, special=None, grow=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    heads, dim, tokens = c.k.shape[2], c.k.shape[3], len(slots)
    rows = torch.randn((tokens, (hq + 2 * heads) * dim + shift), generator=g, device="cuda") * grow
    rows *= torch.exp2(torch.randint(-2, 3, (tokens, 1), generator=g, device="cuda").float())
    rows = rows.to(DTYPES[src])[:, shift:]
    if special:
        special(rows, hq, heads, dim)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in rows.split([hq * dim, heads * dim, heads * dim], 1))
    positions = torch.randint(-50, far, (axes, tokens), generator=g, device="cuda", dtype=I32)
    inv = torch.rand(rot // 2, generator=g, device="cuda") if rot else torch.empty(0, device="cuda")
    axis = torch.randint(-1, axes + 1, (rot // 2,), generator=g, device="cuda", dtype=I32) if axes > 1 else None
    q_out = torch.full((tokens, hq, dim), 3.0, device="cuda", dtype=DTYPES[dtype])
    before = c.copy()
    paged8.gemv_paged8_append(q, k, v, positions if axes > 1 else positions[0], inv, ints(slots), q_out, *c.all, axis=axis,
                              style=style)
    torch.cuda.synchronize()
    turn = lambda x: paged_ref.turned(x.cpu(), positions.cpu(), inv.cpu(), None if axis is None else axis.cpu(), style == "pairs")  # noqa: E731
    # the turn in 32 bits: cos, sin (2 steps each), two products and a sum of values up to 6 * 4 * grow
    slack = 6 * 24 * grow * 2.0 ** -24 if rot else 0.0
    if special is None:
        want = turn(q)
        err = (q_out.double().cpu() - want).abs() - paged_ref.HALF_STEP[DTYPES[dtype]] * want.abs() * 1.001 - slack
        assert not err.numel() or float(err.max()) <= (2.0 ** -25 if dtype == "f16" else 2.0 ** -126), "q"
    held(c, before, slots, turn(k), "k", slack)
    held(c, before, slots, v.double().cpu(), "v", 0.0)


def places(rng, lens, page, pages):
    """Slots of requests of (cached, new) tokens over scattered pages."""
    ids = rng.sample(range(pages), pages)
    slots = []
    for cached, new in lens:
        mine = [ids.pop() for _ in range(-(-(cached + new) // page))]
        slots += [mine[p // page] * page + p % page for p in range(cached, cached + new)]
    return slots


STEPS = {
    "tokens": [(0, 1), (15, 1), (16, 1), (17, 1), (5, 1), (31, 1)],
    "drafts": [(0, 5), (14, 4), (16, 16), (3, 20), (30, 2)],
    "chunks": [(0, 100), (7, 150), (64, 64), (1, 1)],
}


@pytest.mark.parametrize("src", DTYPES)
@pytest.mark.parametrize("code,dtype", KINDS)
@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_append_types(src, code, dtype, style):
    rng = random.Random(1)
    for name, lens in STEPS.items():
        c = Cache(code, 40, 16, 16, 2, 128, seed=len(name))
        run_append(c, src, dtype, places(rng, lens, 16, 40), 4, 128, style=style)


@pytest.mark.parametrize("page,block", [(1, 1), (5, 5), (6, 2), (16, 16), (16, 4), (24, 8), (32, 32), (64, 32), (64, 64), (128, 128), (300, 300),
                                        (1000, 500)])
@pytest.mark.parametrize("dim", [16, 64, 128, 256, 512])
def test_append_blocks(page, block, dim):
    """Blocks of one wave, of several, and of more than four hold; old codes in front of and behind the new ones."""
    rng = random.Random(page + block)
    for name, lens in STEPS.items():
        pages = sum(-(-(c + n) // page) for c, n in lens) + 2
        c = Cache("int8" if block % 2 else "e4m3", pages, page, block, 2, dim, hnd=dim == 64, seed=page)
        run_append(c, "bf16" if dim == 128 else "f32", "bf16", places(rng, lens, page, pages), 2, dim, seed=dim)


@pytest.mark.parametrize("tokens,hq,hkv,dim,rot,axes,style,page,block,hnd", [
    (1, 1, 1, 16, 0, 1, "halves", 1, 1, False), (1, 32, 8, 128, 128, 1, "halves", 16, 16, False), (3, 5, 1, 64, 2, 1, "pairs", 3, 3, True),
    (7, 6, 3, 80, 80, 2, "halves", 24, 8, False), (7, 6, 3, 80, 80, 3, "pairs", 24, 24, True), (5, 4, 4, 64, 50, 3, "halves", 16, 8, True),
    (6, 4, 4, 64, 48, 3, "halves", 5, 1, False), (6, 4, 4, 96, 72, 3, "pairs", 16, 16, False), (2, 2, 1, 512, 512, 1, "halves", 16, 16, True),
    (300, 4, 1, 64, 32, 1, "halves", 16, 16, False), (700, 2, 2, 256, 224, 4, "pairs", 128, 64, True), (0, 4, 1, 64, 64, 1, "halves", 16, 8, False),
    (90, 3, 7, 48, 48, 1, "halves", 32, 16, False), (40, 2, 5, 112, 96, 1, "halves", 8, 8, False)])
@pytest.mark.parametrize("code", ref.CODES)
def test_append_shapes(tokens, hq, hkv, dim, rot, axes, style, page, block, hnd, code):
    rng = random.Random(tokens)
    first = rng.randrange(0, 2 * page)
    pages = -(-(tokens + first) // page) + 2
    slots = places(rng, [(first, tokens)], page, pages)
    if tokens > 4:
        slots[-1], slots[-2] = -1, pages * page  # no place
    c = Cache(code, pages, page, block, hkv, dim, hnd, seed=tokens)
    run_append(c, "f32" if tokens % 2 else "bf16", "bf16" if tokens % 3 else "f16", slots, hq, rot, axes, style, seed=tokens)


@pytest.mark.parametrize("src,shift", [("f32", 1), ("f32", 4), ("f16", 1), ("bf16", 8)])
@pytest.mark.parametrize("code", ref.CODES)
def test_append_unaligned_rows(src, shift, code):
    rng = random.Random(shift)
    c = Cache(code, 20, 16, 16, 2, 64, seed=shift)
    run_append(c, src, "f16", places(rng, STEPS["drafts"], 16, 20), 4, 64, shift=shift)


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("rot", [0, 64, 50])
def test_append_order_within_a_block(code, rot):
    """Tokens of a block in any order, with and without its first place, pages missing behind them."""
    c = Cache(code, 6, 32, 16, 2, 64, seed=3)
    slots = [37, 35, 36, 33, 16, 20, 18, 17, 31, 64, 70, 69, 100, 96, 111, 98, -1, -1, 500]
    run_append(c, "f32", "bf16", slots, 2, rot)


@pytest.mark.parametrize("code", ref.CODES)
def test_append_rows_at_every_scale(code):
    """Values from the least to near the largest floats, a block whose scale grows by any number of steps."""
    for grow in (2.0 ** -140, 2.0 ** -120, 2.0 ** -30, 2.0 ** 30, 2.0 ** 115):
        for byte in ((0, 2), (100, 140), (230, 250)):
            c = Cache(code, 8, 16, 16, 1, 64, seed=5, byte=byte)
            run_append(c, "f32", "bf16", [0, 1, 2, 20, 21, 47, 63], 1, 0, grow=grow)


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("rot", [0, 32, 18])
def test_append_special_values(code, value, rot):
    """A block and head that gets an infinity or NaN is NaN, until the block is begun anew; no other is."""
    c = Cache(code, 4, 16, 16, 2, 64, seed=1)

    def put(rows, hq, heads, dim):
        rows[1, (hq + 1) * dim + 3] = value             # k, head 1, token 1
        rows[2, (hq + heads) * dim + 40] = value        # v, head 0, token 2
    run_append(c, "f32", "bf16", [3, 4, 20, 21], 1, rot, special=put)
    assert c.ks[0, 0].tolist()[1] == 255 and c.vs[1, 0].tolist()[0] == 255
    assert int((c.ks == 255).sum()) == 1 and int((c.vs == 255).sum()) == 1
    run_append(c, "f32", "bf16", [5, 22], 1, rot, seed=2)
    assert c.ks[0, 0].tolist()[1] == 255 and c.vs[1, 0].tolist()[0] == 255
    run_append(c, "f32", "bf16", [0, 16], 1, rot, seed=3)
    assert int((c.ks == 255).sum()) == 0 and int((c.vs == 255).sum()) == 0


@pytest.mark.parametrize("code", ref.CODES)
def test_append_token_by_token(code):
    """A block filled one token at a time with values that grow: within one step of the last scale (int8), and within
    half a step and the smallest one (e4m3), however often the scale grew."""
    c = Cache(code, 1, 64, 64, 1, 64, seed=1)
    x = torch.randn(64, 1, 64, device="cuda") * torch.exp2(torch.arange(64, device="cuda") / 5)[:, None, None]
    out = torch.empty(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, device="cuda")
    for t in range(64):
        paged8.gemv_paged8_append(x[t:t + 1], x[t:t + 1], x[t:t + 1], ints([t]), none, ints([t]), out, *c.all)
    got, want = ref.values(c.k, c.ks)[0], x.double().cpu()
    assert got.equal(ref.values(c.v, c.vs)[0])
    step = 2.0 ** (int(c.ks[0, 0, 0]) - 127)
    assert int(c.ks[0, 0, 0]) == ref.byte_for(float(x.abs().max()), code)
    tol = step if code == "int8" else 2.0 ** -4 * want.abs() + 2.0 ** -9 * step
    assert ((got - want).abs() <= tol).all()


def test_append_same_slot_twice():
    """Either's values, and nothing outside the block."""
    c = Cache("int8", 4, 16, 16, 2, 64, seed=1)
    before = c.copy()
    n = 300
    x = torch.randn(n, 2, 64, device="cuda")
    out = torch.empty(n, 2, 64, device="cuda", dtype=torch.bfloat16)
    paged8.gemv_paged8_append(x, x, x, ints([0] * n), torch.empty(0, device="cuda"), ints([21] * n), out, *c.all)
    for codes, byte, old, old_byte in ((c.k, c.ks, before[0], before[2]), (c.v, c.vs, before[1], before[3])):
        got, old = ref.values(codes, byte), ref.values(old, old_byte)
        assert got[[0, 2, 3]].equal(old[[0, 2, 3]])
        step = ref.scales(byte.cpu())[1, 0]
        near = (got[1, 5] - x.double().cpu()).abs().amin(0)  # of each value, to the nearest token's
        assert (near <= step[:, None] / 2).all()
        rest = [p for p in range(16) if p != 5]
        assert ((got[1, rest] - old[1, rest]).abs() <= step[:, None]).all()


def test_append_interleaved_cache():
    """k and v as the halves of one buffer [page][2][token][head][dim], their scales as well."""
    both = torch.zeros(3, 2, 4, 2, 64, device="cuda", dtype=torch.int8)
    scale = torch.zeros(3, 2, 2, 2, device="cuda", dtype=torch.uint8)
    k, v = torch.randn(2, 1, 2, 64, device="cuda").unbind(0)
    paged8.gemv_paged8_append(k, k, v, ints([0]), torch.empty(0, device="cuda"), ints([6]),
                              torch.empty(1, 2, 64, device="cuda", dtype=torch.float16), both[:, 0], both[:, 1], scale[:, 0], scale[:, 1])
    for i, x in enumerate((k, v)):
        got = both[1, i, 2].double().cpu() * ref.scales(scale[1, i, 1].cpu())[:, None]
        assert ((got - x[0].double().cpu()).abs() <= ref.scales(scale[1, i, 1].cpu())[:, None] / 2).all()
    assert int((scale != 0).sum()) == 4 and not both[0].any() and not both[2].any() and not both[1, :, [0, 1, 3]].any()


def test_append_many_tokens():
    """More tokens than one a workgroup, and than one axis of a grid counts workgroups."""
    for tokens, hkv, dim in ((3001, 2, 64), (2200000, 1, 16)):
        c = Cache("int8", tokens // 16 + 3, 16, 16, hkv, dim, seed=2)
        x = torch.randn(tokens, hkv, dim, device="cuda")
        out = torch.empty(tokens, hkv, dim, device="cuda", dtype=torch.bfloat16)
        slots = torch.arange(5, tokens + 5, device="cuda", dtype=I32)
        paged8.gemv_paged8_append(x, x, x, torch.zeros_like(slots), torch.empty(0, device="cuda"), slots, out, *c.all)
        assert out.equal(x.bfloat16())
        back, back2 = torch.empty_like(x), torch.empty_like(x)
        paged8.gemv_paged8_read(*c.all, slots, back, back2)
        assert back[11:].equal(back2[11:])  # the first block's old scales differ
        blocks = x[11:11 + (tokens - 11) // 16 * 16].unflatten(0, (-1, 16))
        step = torch.exp2(torch.ceil(torch.log2(blocks.abs().amax((1, 3), keepdim=True) / 127)))
        err = (back[11:11 + blocks.shape[0] * 16].unflatten(0, (-1, 16)) - blocks).abs()
        assert (err <= step / 2).all()


# ------------------------------------------------------------------ attention

class Case:
    """Requests of (new tokens, keys), a filled cache, and a scattered table."""

    def __init__(self, lens, code="e4m3", dtype="bf16", hq=4, hkv=2, dim=64, page=16, block=None, hnd=False, seed=0, spare=2,
                 width=None, q_scale=1.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        used = [-(-kv // page) for _, kv in lens]
        ids = torch.randperm(sum(used) + spare, generator=g, device="cuda").tolist()
        width = width or max(used + [1])
        self.table = [[-1] * width for _ in lens]
        at = 0
        for r, u in enumerate(used):
            for j in range(min(u, width)):
                self.table[r][j] = ids[at]
                at += 1
        # values of size about 1: codes about a quarter of their largest
        middle = 127 - (5 if code == "int8" else 7)
        self.c = Cache(code, sum(used) + spare, page, block or page, hkv, dim, hnd, seed + 1, (middle - 1, middle + 2))
        self.starts = [0]
        for n, _ in lens:
            self.starts.append(self.starts[-1] + n)
        self.lens = [kv for _, kv in lens]
        self.q = torch.randn((self.starts[-1], hq, dim), generator=g, device="cuda", dtype=DTYPES[dtype]) * q_scale
        self.scale, self.page = dim ** -0.5, page
        self.window = self.sinks = 0
        self.work = paged.attn_workspace(dim)

    def poison_unused(self):
        """Every place of the cache that holds no key of a request gets a NaN: in e4m3 the place, else the blocks without any."""
        keep = torch.zeros(self.c.k.shape[:2], dtype=torch.bool, device="cuda")
        for row, kv in zip(self.table, self.lens):
            for j in range(kv):
                if j // self.page < len(row) and 0 <= row[j // self.page] < keep.shape[0]:
                    keep[row[j // self.page], j % self.page] = True
        if self.c.code == "e4m3":
            for t in (self.c.k, self.c.v):
                t.view(torch.uint8)[~keep] = 0x7f
        none = ~keep.unflatten(1, (-1, self.c.block)).any(2)
        self.c.ks[none], self.c.vs[none] = 255, 255
        return self

    def run(self, out_dtype=None, workspace="own", out=None, stream=None):
        out = torch.full(self.q.shape, 7.0, device="cuda", dtype=out_dtype or self.q.dtype) if out is None else out
        self.tt, self.qs, self.kl = ints(self.table), ints(self.starts), ints(self.lens)
        torch.cuda.synchronize()
        paged8.gemv_paged8_attn(self.q, *self.c.all, self.tt, self.qs, self.kl, self.scale, out,
                                self.work if isinstance(workspace, str) else workspace, window=self.window, sinks=self.sinks,
                                stream=stream)
        torch.cuda.synchronize()
        return out

    def want(self, out_dtype):
        return ref.attn(self.q, self.c.k, self.c.ks, self.c.v, self.c.vs, ints(self.table, "cpu"), ints(self.starts, "cpu"),
                        ints(self.lens, "cpu"), self.scale, self.window, self.sinks, out_dtype)

    def check(self, out, what=""):
        y, bound, mine = self.want(out.dtype)
        if out.dtype == torch.float16:
            bound = bound + 2.0 ** -25  # below 2^-14 binary16's steps stay 2^-24: half of one, which no share of |y| covers
        got = out.double().cpu()
        assert (got[~mine] == 7.0).all(), f"{what}: a row of no request was written"
        got, y, bound = got[mine], y[mine], bound[mine]
        odd = ~torch.isfinite(y)
        assert torch.isnan(got).equal(torch.isnan(y)), f"{what}: NaN elsewhere"
        assert got[odd & ~torch.isnan(y)].equal(y[odd & ~torch.isnan(y)]), f"{what}: infinities elsewhere"
        err = (got - y).abs()[~odd] - bound[~odd]
        assert not err.numel() or float(err.max()) <= 0, (
            f"{what}: {int((err > 0).sum())} of {err.numel()} values beyond the bound, worst by {float(err.max()):.3e}")


# the first three by tiles of few rows (in the third a request has many of them), the others by tiles of many
LENS = {
    "tokens": [(1, 1), (1, 31), (1, 32), (1, 33), (1, 16), (1, 17), (1, 257), (1, 640)],
    "drafts": [(2, 2), (5, 40), (3, 127), (4, 129), (8, 300), (0, 50), (1, 0), (7, 65)],
    "lone_chunk": [(40, 90)] + [(0, 7)] * 38 + [(1, 300)],
    "chunks": [(64, 64), (33, 100), (1, 5), (130, 130), (17, 400), (0, 0)],
    "before_the_start": [(5, 3), (4, 0), (1, 9), (40, 20)],
    "mixed": [(1, 400), (1, 1), (2, 70), (90, 95)],
}


@pytest.mark.parametrize("code,dtype", KINDS)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_lengths(code, dtype, lens, dim):
    c = Case(LENS[lens], code, dtype, dim=dim).poison_unused()
    c.check(c.run(), lens)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (7, 7), (14, 2), (16, 1), (17, 1), (32, 8), (48, 2), (8, 8)])
@pytest.mark.parametrize("lens", ["tokens", "drafts", "chunks"])
def test_attn_heads(hq, hkv, lens):
    c = Case(LENS[lens], "int8" if hq % 2 else "e4m3", "bf16", hq, hkv, 64, seed=hq).poison_unused()
    c.check(c.run(), f"{hq}/{hkv}")


@pytest.mark.parametrize("page,block", [(1, 1), (2, 1), (7, 7), (8, 8), (16, 2), (16, 8), (16, 16), (24, 8), (24, 24), (24, 6), (32, 16), (33, 11),
                                        (64, 64), (128, 32), (1000, 500)])
@pytest.mark.parametrize("hnd", [False, True])
def test_attn_pages(page, block, hnd):
    for lens in ("tokens", "lone_chunk", "chunks"):
        c = Case(LENS[lens], "int8" if hnd else "e4m3", "f16", page=page, block=block, hnd=hnd, seed=page).poison_unused()
        c.check(c.run(), f"page {page} block {block} {lens}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (32, 0), (33, 4), (100, 40), (64, 64), (5000, 4), (16, 1000)])
@pytest.mark.parametrize("lens", LENS)
def test_attn_window(window, sinks, lens):
    c = Case(LENS[lens], "e4m3" if sinks % 2 else "int8", "bf16" if window % 2 else "f16", seed=window).poison_unused()
    c.window, c.sinks = window, sinks
    c.check(c.run(), f"{window}/{sinks} {lens}")


@pytest.mark.parametrize("code,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_float32_result(code, dtype, dim):
    for lens in ("tokens", "chunks"):
        c = Case(LENS[lens], code, dtype, dim=dim)
        c.check(c.run(torch.float32), f"{code} {dtype} {lens}")


@pytest.mark.parametrize("lens", [[(1, 5000)], [(3, 4001), (1, 9), (1, 2500)], [(20, 3000)], [(1, 3001)] * 5])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_split(lens, dim):
    """Long rows: split over workgroups, with less room for parts, and with none; the counters end as they began; the
    same call gives the same bits."""
    c = Case(lens, "e4m3" if dim == 64 else "int8", "bf16", 8, 2, dim, seed=dim).poison_unused()
    whole = c.run()
    c.check(whole, "split")
    assert c.run().equal(whole)
    assert not c.work[:8192].any()
    few = torch.zeros(8192 + 5 * 16 * (dim + 2) * 4, dtype=torch.uint8, device="cuda")
    c.check(c.run(workspace=few), "room for 5 parts")
    c.check(c.run(workspace=None), "no workspace")
    c.check(c.run(torch.float32), "float32")


def test_attn_one_workspace_for_both_caches():
    """The workspace serves the attention over 16 and over 8 bits in turn."""
    import test_gpu_paged

    for lens in ([(1, 5000)], [(20, 3000)]):
        c, d = Case(lens, "int8", "bf16", 8, 2, 128), test_gpu_paged.Case(lens, "bf16", 8, 2, 128)
        d.work = c.work
        for _ in range(2):
            c.check(c.run(), "8 bits")
            d.check(d.run(), "16 bits")


def test_attn_small_weights_count():
    """One strong key beside 4000 weak ones whose weights together matter: binary16's smallest step must not lose them."""
    c = Case([(1, 4001)], "int8", "f16", 2, 1, 64)
    c.q[:] = 0
    c.q[..., 0] = 8.0
    c.c.k[:] = 0
    c.c.ks[:] = 120
    first = c.table[0][0]
    c.c.ks[first] = 127
    c.c.k[first, 0, 0, 0] = 13  # 13 units of e above the rest: 4000 weights of 2e-6
    c.check(c.run(), "f16")
    c.check(c.run(torch.float32), "f32")


def test_attn_released_pages():
    """Pages behind the window have id -1: never read."""
    lens = [(1, 900), (4, 700), (30, 500)]
    for more in ([], [(0, 1)] * 40):  # by tiles of many rows, and of few
        c = Case(lens + more, "e4m3", "bf16")
        c.window, c.sinks = 100, 4
        for r, (n, kv) in enumerate(lens):
            for j in range(1, (kv - n - 100) // 16):
                c.table[r][j] = -1
        c.check(c.run(), "released")
        for r in range(3):
            c.table[r][0] = -1  # the first tokens too
        c.check(c.run(), "without first tokens")


@pytest.mark.parametrize("page,block", [(3, 1), (16, 8)])
def test_attn_bad_pages(page, block):
    """Ids outside the cache are no keys; a row without keys is zero."""
    for more in ([], [(0, 1)] * 30):
        c = Case([(1, 100), (3, 64), (20, 200), (2, 30)] + more, "int8", "f16", page=page, block=block)
        n = c.c.k.shape[0]
        for row, bad in zip(c.table[:3], (-1, n, 2 ** 31 - 1)):
            row[1] = bad
            row[3] = -2 ** 31
        c.table[3] = [-1] * len(c.table[3])
        out = c.run()
        c.check(out, "bad ids")
        assert not out[24:].any()


def test_attn_narrow_table():
    """Keys past the table's width are not visible."""
    for more in ([], [(0, 1)] * 50):
        c = Case([(1, 100), (2, 20), (40, 90)] + more, "e4m3", "bf16", width=3)
        c.check(c.run(), "narrow")


def test_attn_bad_starts():
    """query_start past the rows is cut; rows outside every request stay as they are."""
    c = Case([(2, 40), (3, 50), (4, 60)], "e4m3", "bf16")
    c.starts = [1, 3, 5, 900]
    c.check(c.run(), "cut")
    c.starts = [0, 2, 2, 6]
    c.check(c.run(), "gaps")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("code", ref.CODES)
def test_attn_nan_blocks_reach_only_their_rows(dim, code):
    """A block whose scale is NaN changes the rows that see one of its keys and no other."""
    for what in ("ks", "vs"):
        for window in (0, 9):
            for more in ([], [(0, 1)] * 60):
                c = Case([(20, 50), (1, 40), (40, 70)] + more, code, "bf16", dim=dim, block=8, seed=3)
                c.window, c.sinks = window, 2
                t = getattr(c.c, what)
                for r, j in ((0, 41), (1, 3), (2, 55)):
                    t[c.table[r][j // 16], j % 16 // 8, 1] = 255
                c.check(c.run(), f"NaN in {what}, window {window}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_values_past_binary16(dim):
    """Values beyond binary16's range are its infinities there, for the rows that see them."""
    for lens in ([(20, 50), (1, 40), (40, 70)], [(1, 40), (1, 70), (2, 50), (1, 9)]):
        c = Case(lens, "int8", "f16", dim=dim, block=8, seed=3)
        for r, j in ((0, 30), (1, 3)):
            at = c.table[r][j // 16], j % 16 // 8, 1
            c.c.vs[at] = 127 + 13
            c.c.v[at[0], at[1] * 8:at[1] * 8 + 8, 1] = 9 - 2 * r * 9  # 9 2^13 and its negative
        c.check(c.run(), "past the range")


def test_attn_equal_and_huge_scores():
    for lens in ([(1, 100), (4, 33)], [(1, 100), (40, 133)]):
        c = Case(lens, "int8", "bf16")
        c.c.k[:] = 0
        c.check(c.run(), "equal")
        c = Case(lens, "e4m3", "f16", q_scale=300.0)
        c.check(c.run(), "huge")
        c.scale = -c.scale
        c.check(c.run(), "negative scale")
        c.scale = 0.0
        c.check(c.run(), "zero scale")


def test_attn_strides():
    """q as a part of a qkv row, heads apart; out with rows and heads apart; caches as halves of one buffer; scales with
    any strides."""
    for lens in ("chunks", "tokens"):
        c = Case(LENS[lens], "int8", "bf16", 4, 2, 64)
        rows = torch.randn(c.q.shape[0], 10, 64, device="cuda", dtype=torch.bfloat16)
        rows[:, 1:9:2] = c.q
        c.q = rows[:, 1:9:2]
        both = torch.stack([c.c.k, c.c.v], 1).contiguous()
        c.c.k, c.c.v = both[:, 0], both[:, 1]
        far = torch.full((*c.c.ks.shape, 5), 255, dtype=torch.uint8, device="cuda")
        far[..., 2], far[..., 4] = c.c.ks, c.c.vs
        c.c.ks, c.c.vs = far[..., 2], far[..., 4]
        wide = torch.full((6, c.q.shape[0], 72), 7.0, device="cuda", dtype=torch.bfloat16)
        c.check(c.run(out=wide[1:5, :, :64].transpose(0, 1)), "strides")
        assert (wide[0] == 7).all() and (wide[5] == 7).all() and (wide[:, :, 64:] == 7).all()


def test_far_pages():
    """A cache of more than 2^32 bytes, its last pages written, read and attended to."""
    pages = 2 ** 32 // (16 * 8 * 128) + 40
    c = Case([(1, 100), (5, 60)], "int8", "bf16", 16, 8, 128)
    k, v = (torch.empty((pages, 16, 8, 128), device="cuda", dtype=torch.int8) for _ in "kv")
    ks, vs = (torch.empty((pages, 1, 8), device="cuda", dtype=torch.uint8) for _ in "kv")
    small = c.c.k.shape[0]
    k[-small:], v[-small:], ks[-small:], vs[-small:] = c.c.k, c.c.v, c.c.ks, c.c.vs
    x = torch.randn(3, 8, 128, device="cuda", dtype=torch.bfloat16)
    near, far = ints([small * 16 - 3, small * 16 - 2, 4]), ints([pages * 16 - 3, pages * 16 - 2, (pages - small) * 16 + 4])
    out, none = torch.empty_like(x), torch.empty(0, device="cuda")
    paged8.gemv_paged8_append(x, x, x, ints([0] * 3), none, near, out, *c.c.all)
    paged8.gemv_paged8_append(x, x, x, ints([0] * 3), none, far, out, k, v, ks, vs)
    assert k[-small:].equal(c.c.k) and v[-small:].equal(c.c.v) and ks[-small:].equal(c.c.ks) and vs[-small:].equal(c.c.vs)
    a, b = torch.empty_like(x), torch.empty_like(x)
    paged8.gemv_paged8_read(*c.c.all, near, a)
    paged8.gemv_paged8_read(k, v, ks, vs, far, b)
    assert a.equal(b)
    y, bound, _ = c.want(torch.bfloat16)
    table = torch.full((2, 20), -1, dtype=I32, device="cuda")
    table[:, 3:3 + len(c.table[0])] = ints(c.table) + (pages - small)
    out = torch.empty_like(c.q)
    paged8.gemv_paged8_attn(c.q, k, v, ks, vs, table[:, 3:3 + len(c.table[0])], ints(c.starts), ints(c.lens), c.scale, out, c.work)
    assert ((out.double().cpu() - y).abs() <= bound).all()


@pytest.mark.parametrize("new", [(0, 1, 1, 1, 3), (0, 1, 9, 30)])
def test_attn_many_requests(new):
    rng = random.Random(5)
    c = Case([(rng.choice(new), rng.randrange(0, 50)) for _ in range(600)], "int8", "f16", 2, 1, 64)
    c.check(c.run(), "600 requests")


# ------------------------------------------------------------------ streams and graphs

def test_attn_on_another_stream():
    c = Case([(1, 2000), (9, 300)], "e4m3", "bf16")
    side = torch.cuda.Stream()
    c.check(c.run(stream=side), "side stream")
    with torch.cuda.stream(side):
        c.check(c.run(), "current stream")


@pytest.mark.parametrize("code", ref.CODES)
def test_step_in_a_graph(code):
    """Slots, append, attention and reading of one step captured once and replayed for new lengths, eager work between."""
    requests, tokens, page, hq, hkv, dim, pages = 3, 12, 16, 4, 2, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    cached, fresh = ints([0] * requests), ints([0] * requests)
    table = torch.full((requests, 16), -1, dtype=I32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").int()
    new = lambda n: torch.zeros(n, dtype=I32, device="cuda")  # noqa: E731
    qs, kl, tr, pos, slots, used = new(requests + 1), new(requests), new(tokens), new(tokens), new(tokens), new(1)
    cache = paged8.cache(pages, page, hkv, dim, code, block=8)
    rows = torch.randn(tokens, (hq + 2 * hkv) * dim, generator=g, device="cuda")
    q, k, v = (t.unflatten(1, (-1, dim)) for t in rows.split([hq * dim, hkv * dim, hkv * dim], 1))
    inv = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    q_out, out = (torch.zeros(tokens, hq, dim, device="cuda", dtype=torch.bfloat16) for _ in "qo")
    back = torch.zeros(2, tokens, hkv, dim, device="cuda", dtype=torch.bfloat16)
    work = paged.attn_workspace(dim)

    def step():
        paged.gemv_paged_slots(cached, fresh, free, page, table, qs, kl, tr, pos, slots, used)
        paged8.gemv_paged8_append(q, k, v, pos, inv, slots, q_out, *cache)
        paged8.gemv_paged8_attn(q_out, *cache, table, qs, kl, 0.125, out, work)
        paged8.gemv_paged8_read(*cache, slots, back[0], back[1])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state = (*cache, table)
    bytes_ = lambda t: t.view(torch.uint8) if t.dtype != I32 else t  # noqa: E731
    for n, f in enumerate(([5, 1, 4], [1, 1, 1], [2, 0, 9], [1, 7, 1], [3, 3, 3])):
        fresh.copy_(ints(f))
        rows.copy_(torch.randn(rows.shape, generator=g, device="cuda") * (1 + n))
        before = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        first = [bytes_(t).clone() for t in (*state, slots)] + [out[:sum(f)].clone(), back.clone()]
        assert float(first[-2].abs().sum()) > 0
        for t, b in zip(state, before):
            bytes_(t).copy_(bytes_(b))
        step()
        torch.cuda.synchronize()
        for a, b in zip(first, [bytes_(t) for t in (*state, slots)] + [out[:sum(f)], back]):
            assert a.equal(b), f"replay {n}"
        y, bound, _ = ref.attn(q_out[:sum(f)], cache[0], cache[2], cache[1], cache[3], table, qs, kl, 0.125, 0, 0, torch.bfloat16)
        assert ((out[:sum(f)].double().cpu() - y).abs() <= bound).all()
        at = slots[:sum(f)].cpu().long()
        for i in range(2):
            want = ref.values(cache[i], cache[2 + i]).flatten(0, 1)[at]
            assert back[i, :sum(f)].cpu().equal(want.bfloat16()) and not back[i, sum(f):].any()
        cached.copy_(kl)
        free.copy_(torch.roll(free, -int(used)))  # the captured address; its used ids move to the end


def test_two_graphs_with_a_workspace_each():
    """Two captured calls on streams of their own, replayed at once, each with its own workspace."""
    cases = [Case([(1, 5000), (1, 700)], "int8", "bf16", 8, 2, 128, seed=s) for s in (1, 2)]
    graphs = []
    for c in cases:
        c.out = c.run()
        c.graph_out = torch.empty_like(c.out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            paged8.gemv_paged8_attn(c.q, *c.c.all, c.tt, c.qs, c.kl, c.scale, c.graph_out, c.work)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, graph, stream in zip(cases, graphs, streams):
            with torch.cuda.stream(stream):
                c.graph_out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for c in cases:
            assert c.graph_out.equal(c.out)
