"""The paged operators on the GPU against the 64-bit references of paged_ref:
lengths, head layouts, types, strides, page sizes and masks where they can go
wrong, and what they promise about buffers, streams and graphs."""
import random

import pytest
import torch

import paged_ref
from decode_gemv_elementwise_amd import paged

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
I32 = torch.int32


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=I32, device=device)


# ------------------------------------------------------------------ slots

def run_slots(cached, fresh, free, page, table, tokens):
    n = len(cached)
    t = ints(table)
    out = {"block_table": t, "query_start": ints([-7] * (n + 1)), "kv_len": ints([-7] * n),
           "token_request": ints([-7] * tokens), "positions": ints([-7] * tokens), "slots": ints([-7] * tokens),
           "used": ints([-7])}
    paged.gemv_paged_slots(ints(cached), ints(fresh), ints(free), page, t, out["query_start"], out["kv_len"],
                           out["token_request"], out["positions"], out["slots"], out["used"])
    torch.cuda.synchronize()
    return {k: v.cpu().tolist() for k, v in out.items()}


SLOTS = {
    "one": ([0], [1], 16, 4, 1, 9),
    "first_token_of_a_page": ([16, 15, 17], [1, 1, 1], 16, 4, 3, 9),
    "nothing_new": ([5, 0, 33], [0, 0, 0], 16, 4, 0, 9),
    "padded": ([5, 0, 33], [2, 0, 40], 16, 6, 600, 9),
    "negative_lengths": ([-3, 4, 7], [5, -2, 1], 4, 4, 8, 9),
    "capacity_cuts": ([3, 9, 0, 5], [4, 9, 300, 5], 8, 60, 200, 60),
    "no_free_page": ([15, 16, 16], [3, 2, 1], 16, 4, 6, 1),
    "narrow_table": ([30, 3], [10, 2], 4, 8, 12, 9),
    "page_of_one": ([3, 0, 2], [2, 4, 0], 1, 8, 7, 9),
    "long_chunk": ([7], [5000], 24, 300, 5000, 300),
}


@pytest.mark.parametrize("name", SLOTS)
def test_slots(name):
    cached, fresh, page, width, tokens, nfree = SLOTS[name]
    rng = random.Random(name)
    free = rng.sample(range(5000), nfree)
    table = [[rng.randrange(5000, 9000) for _ in range(width)] for _ in cached]
    got = run_slots(cached, fresh, free, page, table, tokens)
    assert got == paged_ref.slots(cached, fresh, free, page, table, tokens)


@pytest.mark.parametrize("requests", [1, 63, 64, 65, 255, 256, 1023, 1024, 1025, 4100])
def test_slots_many_requests(requests):
    rng = random.Random(requests)
    cached = [rng.choice([0, rng.randrange(0, 200)]) for _ in range(requests)]
    fresh = [rng.choice([0, 1, 1, rng.randrange(0, 60)]) for _ in range(requests)]
    tokens = sum(fresh) + rng.choice([0, 300])
    free = rng.sample(range(100000), sum(fresh) + requests)
    table = [[rng.randrange(100000, 200000) for _ in range(17)] for _ in range(requests)]
    got = run_slots(cached, fresh, free, 16, table, tokens)
    assert got == paged_ref.slots(cached, fresh, free, 16, table, tokens)


def test_slots_drops_bad_entries():
    """A table entry that is negative, or whose slot passes 2^31 - 1, gives slot -1."""
    got = run_slots([1, 1, 1], [1, 1, 1], [], 16, [[-1], [2 ** 31 - 1], [2 ** 27 - 1]], 3)
    assert got["slots"] == [-1, -1, 2 ** 31 - 16 + 1]


def test_slots_strided_table():
    wide = torch.full((3, 10), 77, dtype=I32, device="cuda")
    table = wide[:, 2:6]
    one = lambda n: torch.empty(n, dtype=I32, device="cuda")  # noqa: E731
    slots = one(4)
    paged.gemv_paged_slots(ints([0, 3, 4]), ints([1, 1, 2]), ints([5, 6, 7]), 4, table, one(4), one(3), one(4), one(4),
                           slots, one(1))
    assert slots.tolist() == [20, 77 * 4 + 3, 24, 25]
    want = torch.full((3, 10), 77)
    want[0, 2], want[2, 3] = 5, 6
    assert wide.cpu().equal(want.int())


# ------------------------------------------------------------------ append

def close(got, want, dtype, slack, what):
    """got, rounded once to dtype, against want: half a step, and `slack` times 2^-24 of the terms for the 32-bit turn."""
    err = (got.double().cpu() - want).abs()
    tol = paged_ref.HALF_STEP[dtype] * want.abs() * 1.001 + slack
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((err - tol).max()):.3e}"


def run_append(src, dtype, tokens, hq, hkv, dim, rot, axes, style, page, hnd=False, shift=0, far=100000, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = (hq + 2 * hkv) * dim + shift
    rows = torch.randn((tokens, width), generator=g, device="cuda", dtype=DTYPES[src])[:, shift:]
    q, k, v = (t.unflatten(1, (-1, dim)) for t in rows.split([hq * dim, hkv * dim, hkv * dim], 1))
    positions = torch.randint(-50, far, (axes, tokens), generator=g, device="cuda", dtype=I32)
    inv = torch.rand(rot // 2, generator=g, device="cuda") if rot else torch.empty(0, device="cuda")
    axis = torch.randint(-1, axes + 1, (rot // 2,), generator=g, device="cuda", dtype=I32) if axes > 1 else None
    pages = -(-tokens // page) + 2
    shape = (pages, hkv, page, dim) if hnd else (pages, page, hkv, dim)
    kc, vc = (torch.full(shape, 3.0, device="cuda", dtype=DTYPES[dtype]) for _ in "kv")
    if hnd:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].int()
    if tokens > 4:
        slots[1], slots[3] = -1, pages * page  # no place
    q_out = torch.full((tokens, hq, dim), 3.0, device="cuda", dtype=DTYPES[dtype])
    paged.gemv_paged_append(q, k, v, positions if axes > 1 else positions[0], inv, slots, q_out, kc, vc, axis=axis,
                            style=style)
    torch.cuda.synchronize()
    pairs = style == "pairs"
    # the turn in 32 bits: cos, sin (2 steps each), two products and a sum of values up to 6
    slack = 6 * 6 * 2.0 ** -24 if rot else 0.0
    turn = lambda x: paged_ref.turned(x.cpu(), positions.cpu(), inv.cpu(), None if axis is None else axis.cpu(), pairs)  # noqa: E731
    close(q_out, turn(q), DTYPES[dtype], slack, "q")
    want_k, want_v = torch.full(kc.shape, 3.0).double(), torch.full(vc.shape, 3.0).double()
    tk = turn(k)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, s % page], want_v[s // page, s % page] = tk[t], v[t].double().cpu()
    close(kc, want_k, DTYPES[dtype], slack, "k")
    close(vc, want_v, DTYPES[dtype], 0.0, "v")


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_append_types(src, dtype, style):
    run_append(src, dtype, 9, 8, 2, 128, 128, 1, style, 16)


@pytest.mark.parametrize("tokens,hq,hkv,dim,rot,axes,style,page,hnd", [
    (1, 1, 1, 8, 0, 1, "halves", 1, False), (1, 32, 8, 128, 128, 1, "halves", 16, False),
    (3, 5, 1, 64, 2, 1, "pairs", 3, True), (7, 6, 3, 72, 72, 2, "halves", 24, False), (7, 6, 3, 72, 72, 3, "pairs", 24, True),
    (5, 4, 4, 64, 50, 3, "halves", 16, True), (6, 4, 4, 64, 48, 3, "halves", 5, False), (2, 2, 1, 512, 512, 1, "halves", 16, True),
    (300, 4, 1, 64, 32, 1, "halves", 16, False), (700, 2, 2, 256, 224, 4, "pairs", 128, True), (0, 4, 1, 64, 64, 1, "halves", 16, False)])
def test_append_shapes(tokens, hq, hkv, dim, rot, axes, style, page, hnd):
    run_append("f32" if tokens % 2 else "bf16", "bf16" if tokens % 3 else "f16", tokens, hq, hkv, dim, rot, axes, style,
               page, hnd, seed=tokens)


@pytest.mark.parametrize("src,shift", [("f32", 1), ("f32", 4), ("f16", 1), ("bf16", 8)])
def test_append_unaligned_rows(src, shift):
    run_append(src, "f16", 6, 4, 2, 64, 64, 1, "halves", 16, shift=shift)


def test_append_far_positions():
    """A position of 2^31 - 1 keeps its fraction of a turn."""
    run_append("f32", "f16", 12, 2, 1, 64, 64, 1, "halves", 16, far=2 ** 31 - 1)


def test_append_special_values_pass():
    q = torch.zeros(2, 1, 64, device="cuda")
    q[0, 0, 3], q[1, 0, 40] = float("inf"), float("nan")
    kc, vc = (torch.zeros(1, 4, 1, 64, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    out = torch.empty(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    paged.gemv_paged_append(q, q, q, ints([0, 0]), torch.ones(8, device="cuda"), ints([0, 2]), out, kc, vc)
    assert torch.isinf(out[0, 0, 3]) and torch.isnan(out[1, 0, 40]) and int(torch.isnan(out[1]).sum()) == 1
    assert torch.isinf(vc[0, 0, 0, 3]) and torch.isnan(vc[0, 2, 0, 40]) and not vc[0, 1].any() and not vc[0, 3].any()


def test_append_interleaved_cache():
    """k and v as the halves of one buffer [page][2][token][head][dim]."""
    both = torch.zeros(3, 2, 4, 2, 64, device="cuda", dtype=torch.float16)
    k, v = torch.randn(2, 1, 2, 64, device="cuda").unbind(0)
    paged.gemv_paged_append(k, k, v, ints([0]), torch.empty(0, device="cuda"), ints([6]),
                            torch.empty(1, 2, 64, device="cuda", dtype=torch.float16), both[:, 0], both[:, 1])
    assert both[1, 0, 2].equal(k[0].half()) and both[1, 1, 2].equal(v[0].half())
    assert int((both != 0).sum()) == int((k.half() != 0).sum() + (v.half() != 0).sum())


# ------------------------------------------------------------------ attention

class Case:
    """Requests of (new tokens, keys), a filled cache, and a scattered table."""

    def __init__(self, lens, dtype="bf16", hq=4, hkv=2, dim=64, page=16, hnd=False, seed=0, spare=2, width=None, q_scale=1.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = DTYPES[dtype]
        used = [-(-kv // page) for _, kv in lens]
        ids = torch.randperm(sum(used) + spare, generator=g, device="cuda").tolist()
        width = width or max(used + [1])
        self.table = [[-1] * width for _ in lens]
        at = 0
        for r, u in enumerate(used):
            for j in range(min(u, width)):
                self.table[r][j] = ids[at]
                at += 1
        pages = sum(used) + spare
        shape = (pages, hkv, page, dim) if hnd else (pages, page, hkv, dim)
        self.k, self.v = (torch.randn(shape, generator=g, device="cuda", dtype=dt) for _ in "kv")
        if hnd:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.starts = [0]
        for n, _ in lens:
            self.starts.append(self.starts[-1] + n)
        self.lens = [kv for _, kv in lens]
        self.q = torch.randn((self.starts[-1], hq, dim), generator=g, device="cuda", dtype=dt) * q_scale
        self.scale, self.page = dim ** -0.5, page
        self.window = self.sinks = 0
        self.work = paged.attn_workspace(dim)

    def poison_unused(self):
        """Every place of the cache that holds no key of a request gets a NaN."""
        keep = torch.zeros(self.k.shape[:2], dtype=torch.bool, device="cuda")
        for row, kv in zip(self.table, self.lens):
            for j in range(kv):
                if j // self.page < len(row) and 0 <= row[j // self.page] < keep.shape[0]:
                    keep[row[j // self.page], j % self.page] = True
        self.k[~keep], self.v[~keep] = float("nan"), float("nan")
        return self

    def run(self, out_dtype=None, workspace="own", out=None, stream=None):
        out = torch.full(self.q.shape, 7.0, device="cuda", dtype=out_dtype or self.q.dtype) if out is None else out
        self.tt, self.qs, self.kl = ints(self.table), ints(self.starts), ints(self.lens)
        torch.cuda.synchronize()
        paged.gemv_paged_attn(self.q, self.k, self.v, self.tt, self.qs, self.kl, self.scale, out,
                              self.work if isinstance(workspace, str) else workspace, window=self.window,
                              sinks=self.sinks, stream=stream)
        torch.cuda.synchronize()
        return out

    def check(self, out, what=""):
        y, bound, mine = paged_ref.attn(self.q, self.k, self.v, ints(self.table, "cpu"), ints(self.starts, "cpu"),
                                        ints(self.lens, "cpu"), self.scale, self.window, self.sinks, out.dtype)
        got = out.double().cpu()
        assert (got[~mine] == 7.0).all(), f"{what}: a row of no request was written"
        got, y, bound = got[mine], y[mine], bound[mine]
        odd = ~torch.isfinite(y)
        assert torch.isnan(got).equal(torch.isnan(y)), f"{what}: NaN elsewhere"
        assert got[odd & ~torch.isnan(y)].equal(y[odd & ~torch.isnan(y)]), f"{what}: infinities elsewhere"
        err = (got - y).abs()[~odd] - bound[~odd]
        assert not err.numel() or float(err.max()) <= 0, (
            f"{what}: {int((err > 0).sum())} of {err.numel()} values beyond the bound, worst by {float(err.max()):.3e}")


LENS = {
    "tokens": [(1, 1), (1, 31), (1, 32), (1, 33), (1, 16), (1, 17), (1, 257), (1, 640)],
    "drafts": [(2, 2), (5, 40), (3, 127), (4, 129), (8, 300), (0, 50), (1, 0), (7, 65)],
    "chunks": [(64, 64), (33, 100), (1, 5), (130, 130), (17, 400), (0, 0)],
    "before_the_start": [(5, 3), (4, 0), (1, 9), (40, 20)],
}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_lengths(dtype, lens, dim):
    c = Case(LENS[lens], dtype, dim=dim).poison_unused()
    c.check(c.run(), lens)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (7, 7), (14, 2), (16, 1), (17, 1), (32, 8), (48, 2), (8, 8)])
@pytest.mark.parametrize("lens", ["drafts", "chunks"])
def test_attn_heads(hq, hkv, lens):
    c = Case(LENS[lens], "bf16", hq, hkv, 64, seed=hq).poison_unused()
    c.check(c.run(), f"{hq}/{hkv}")


@pytest.mark.parametrize("page", [1, 2, 7, 8, 16, 24, 32, 33, 64, 128, 1000])
@pytest.mark.parametrize("hnd", [False, True])
def test_attn_pages(page, hnd):
    for lens in ("tokens", "chunks"):
        c = Case(LENS[lens], "f16", page=page, hnd=hnd, seed=page).poison_unused()
        c.check(c.run(), f"page {page} {lens}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (32, 0), (33, 4), (100, 40), (64, 64), (5000, 4), (16, 1000)])
@pytest.mark.parametrize("lens", LENS)
def test_attn_window(window, sinks, lens):
    c = Case(LENS[lens], "bf16" if window % 2 else "f16", seed=window).poison_unused()
    c.window, c.sinks = window, sinks
    c.check(c.run(), f"{window}/{sinks} {lens}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_float32_result(dtype, dim):
    for lens in ("tokens", "chunks"):
        c = Case(LENS[lens], dtype, dim=dim)
        c.check(c.run(torch.float32), f"{dtype} {lens}")


@pytest.mark.parametrize("lens", [[(1, 5000)], [(3, 4001), (1, 9), (1, 2500)], [(20, 3000)], [(1, 3001)] * 5])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_split(lens, dim):
    """Long rows: split over workgroups, with less room for parts, and with none; the counters end as they began; the
    same call gives the same bits."""
    c = Case(lens, "bf16", 8, 2, dim, seed=dim).poison_unused()
    whole = c.run()
    c.check(whole, "split")
    assert c.run().equal(whole)
    assert not c.work[:8192].any()
    few = torch.zeros(8192 + 5 * 16 * (dim + 2) * 4, dtype=torch.uint8, device="cuda")
    c.check(c.run(workspace=few), "room for 5 parts")
    c.check(c.run(workspace=None), "no workspace")
    c.check(c.run(torch.float32), "float32")


def test_attn_small_weights_count():
    """One strong key beside 4000 weak ones whose weights together matter: binary16's smallest step must not lose them."""
    c = Case([(1, 4001)], "f16", 2, 1, 64)
    c.q[:] = 0
    c.q[..., 0] = 8.0
    k = torch.zeros_like(c.k)
    k[c.table[0][0], 0, 0, 0] = 13.0  # 13 units of e above the rest: 4000 weights of 2e-6
    c.k = k
    c.check(c.run(), "f16")
    c.check(c.run(torch.float32), "f32")


def test_attn_released_pages():
    """Pages behind the window have id -1: never read."""
    c = Case([(1, 900), (4, 700), (30, 500)], "bf16")
    c.window, c.sinks = 100, 4
    for r, (n, kv) in enumerate([(1, 900), (4, 700), (30, 500)]):
        for j in range(1, (kv - n - 100) // 16):
            c.table[r][j] = -1
    c.check(c.run(), "released")
    for r in range(3):
        c.table[r][0] = -1  # the first tokens too
    c.check(c.run(), "without first tokens")


@pytest.mark.parametrize("page", [3, 16])
def test_attn_bad_pages(page):
    """Ids outside the cache are no keys; a row without keys is zero."""
    c = Case([(1, 100), (3, 64), (20, 200), (2, 30)], "f16", page=page)
    n = c.k.shape[0]
    for row, bad in zip(c.table, (-1, n, 2 ** 31 - 1)):
        row[1] = bad
        row[3] = -2 ** 31
    c.table[3] = [-1] * len(c.table[3])
    out = c.run()
    c.check(out, "bad ids")
    assert not out[24:].any()


def test_attn_narrow_table():
    """Keys past the table's width are not visible."""
    c = Case([(1, 100), (2, 20), (40, 90)], "bf16", width=3)
    c.check(c.run(), "narrow")


def test_attn_bad_starts():
    """query_start past the rows is cut; rows outside every request stay as they are."""
    c = Case([(2, 40), (3, 50), (4, 60)], "bf16")
    c.starts = [1, 3, 5, 900]
    c.check(c.run(), "cut")
    c.starts = [0, 2, 2, 6]
    c.check(c.run(), "gaps")


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attn_special_values_reach_only_their_rows(value, dim):
    """A key that holds an infinity or NaN changes the rows that see it and no other."""
    for what in ("k", "v"):
        for window in (0, 9):
            c = Case([(20, 50), (1, 40), (40, 70)], "bf16", dim=dim, seed=3)
            c.window, c.sinks = window, 2
            t = getattr(c, what)
            for r, j in ((0, 41), (1, 3), (2, 55)):
                t[c.table[r][j // 16], j % 16, 1, 5] = value
            if what == "k":
                c.q[..., 5] = c.q[..., 5].abs() + 0.5  # no 0 * inf, one sign
            c.check(c.run(), f"{value} in {what}, window {window}")


def test_attn_equal_and_huge_scores():
    c = Case([(1, 100), (4, 33)], "bf16")
    c.k[:] = 0
    c.check(c.run(), "equal")
    c = Case([(1, 100), (4, 33)], "f16", q_scale=300.0)
    c.check(c.run(), "huge")
    c.scale = -c.scale
    c.check(c.run(), "negative scale")
    c.scale = 0.0
    c.check(c.run(), "zero scale")


def test_attn_strides():
    """q as a part of a qkv row, heads apart; out with rows and heads apart; caches as halves of one buffer."""
    c = Case(LENS["chunks"], "bf16", 4, 2, 64)
    rows = torch.randn(c.q.shape[0], 10, 64, device="cuda", dtype=torch.bfloat16)
    rows[:, 1:9:2] = c.q
    c.q = rows[:, 1:9:2]
    both = torch.stack([c.k, c.v], 1).contiguous()
    c.k, c.v = both[:, 0], both[:, 1]
    wide = torch.full((6, c.q.shape[0], 72), 7.0, device="cuda", dtype=torch.bfloat16)
    c.check(c.run(out=wide[1:5, :, :64].transpose(0, 1)), "strides")
    assert (wide[0] == 7).all() and (wide[5] == 7).all() and (wide[:, :, 64:] == 7).all()


def test_attn_strided_table_and_far_pages():
    """Table rows apart; a cache of more than 2^31 elements, its last pages used."""
    pages = 2 ** 31 // (16 * 8 * 128) + 40
    c = Case([(1, 100), (5, 60)], "bf16", 16, 8, 128)
    k, v = (torch.empty((pages, 16, 8, 128), device="cuda", dtype=torch.bfloat16) for _ in "kv")
    small = c.k.shape[0]
    k[-small:], v[-small:] = c.k, c.v
    y, bound, _ = paged_ref.attn(c.q, c.k, c.v, ints(c.table, "cpu"), ints(c.starts, "cpu"), ints(c.lens, "cpu"), c.scale,
                                 0, 0, torch.bfloat16)
    table = torch.full((2, 20), -1, dtype=I32, device="cuda")
    table[:, 3:3 + len(c.table[0])] = ints(c.table) + (pages - small)
    out = torch.empty_like(c.q)
    paged.gemv_paged_attn(c.q, k, v, table[:, 3:3 + len(c.table[0])], ints(c.starts), ints(c.lens), c.scale, out, c.work)
    assert ((out.double().cpu() - y).abs() <= bound).all()


def test_attn_many_requests():
    rng = random.Random(5)
    c = Case([(rng.choice([0, 1, 1, 1, 3]), rng.randrange(0, 50)) for _ in range(600)], "f16", 2, 1, 64)
    c.check(c.run(), "600 requests")


# ------------------------------------------------------------------ streams and graphs

def test_attn_on_another_stream():
    c = Case([(1, 2000), (9, 300)], "bf16")
    side = torch.cuda.Stream()
    c.check(c.run(stream=side), "side stream")
    with torch.cuda.stream(side):
        c.check(c.run(), "current stream")


def test_step_in_a_graph():
    """Slots, append and attention of one step captured once and replayed for new lengths, eager work between."""
    requests, tokens, page, hq, hkv, dim, pages = 3, 12, 16, 4, 2, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    cached, fresh = ints([0] * requests), ints([0] * requests)
    table = torch.full((requests, 16), -1, dtype=I32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").int()
    new = lambda n: torch.zeros(n, dtype=I32, device="cuda")  # noqa: E731
    qs, kl, tr, pos, slots, used = new(requests + 1), new(requests), new(tokens), new(tokens), new(tokens), new(1)
    kc, vc = (torch.zeros(pages, page, hkv, dim, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    rows = torch.randn(tokens, (hq + 2 * hkv) * dim, generator=g, device="cuda")
    q, k, v = (t.unflatten(1, (-1, dim)) for t in rows.split([hq * dim, hkv * dim, hkv * dim], 1))
    inv = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    q_out, out = (torch.zeros(tokens, hq, dim, device="cuda", dtype=torch.bfloat16) for _ in "qo")
    work = paged.attn_workspace(dim)

    def step():
        paged.gemv_paged_slots(cached, fresh, free, page, table, qs, kl, tr, pos, slots, used)
        paged.gemv_paged_append(q, k, v, pos, inv, slots, q_out, kc, vc)
        paged.gemv_paged_attn(q_out, kc, vc, table, qs, kl, 0.125, out, work)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    taken = 0
    for n, f in enumerate(([5, 1, 4], [1, 1, 1], [2, 0, 9], [1, 7, 1], [3, 3, 3])):
        fresh.copy_(ints(f))
        rows.copy_(torch.randn(rows.shape, generator=g, device="cuda"))
        before = (kc.clone(), vc.clone(), table.clone())
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in (out[:sum(f)], kc, vc, table, slots)]
        assert float(first[0].abs().sum()) > 0
        kc.copy_(before[0]), vc.copy_(before[1]), table.copy_(before[2])
        step()
        torch.cuda.synchronize()
        for a, b in zip(first, (out[:sum(f)], kc, vc, table, slots)):
            assert a.equal(b), f"replay {n}"
        y, bound, _ = paged_ref.attn(q_out[:sum(f)], kc, vc, table, qs, kl, 0.125, 0, 0, torch.bfloat16)
        assert ((out[:sum(f)].double().cpu() - y).abs() <= bound).all()
        cached.copy_(kl)
        free = free  # the captured address; its used ids move to the end
        free.copy_(torch.roll(free, -int(used)))
        taken += int(used)
    assert taken <= pages
