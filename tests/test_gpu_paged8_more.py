"""The operators over a paged cache in 8 bits: tiles that shares cut, tiles of several
heads, the plan's coarse units, far strides, any order of calls, and the calls' two ways
through the binding."""
import random
import sys

import pytest
import torch

import decode_gemv_elementwise_amd as package
import paged8_ref as ref
from decode_gemv_elementwise_amd import binding, paged, paged8
from test_gpu_paged8 import I32, KINDS, Cache, Case, ints, places, run_append

pytestmark = pytest.mark.gpu

COUNTERS = 8192  # bytes at the workspace's start


def check_twice(c, what):
    """Right, the same bits again, and the counters as they were."""
    out = c.run()
    c.check(out, what)
    assert c.run().equal(out), f"{what}: another result the second time"
    assert not c.work[:COUNTERS].any(), f"{what}: counters left"
    return out


@pytest.mark.parametrize("code,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(9, 5000)], [(40, 3000)], [(17, 4097), (1, 3000), (130, 1500)], [(33, 2000)] * 3])
def test_cut_tiles(lens, dim, code, dtype):
    """Few tiles over many keys: every tile is cut over many workgroups and joined."""
    c = Case(lens, code, dtype, 4, 2, dim, seed=dim).poison_unused()
    check_twice(c, f"{lens} {dim}")
    c.check(c.run(torch.float32), "float32")


@pytest.mark.parametrize("page,block", [(1, 1), (8, 4), (12, 12), (16, 1), (16, 2), (16, 8), (24, 8), (48, 16), (48, 24), (64, 4), (64, 32), (96, 48)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_of_long_chunks(page, block, dim):
    """Both ways to find a block's keys, by tiles of many rows and of few."""
    for more in ([], [(0, 3)] * 100):
        c = Case([(20, 700), (70, 333), (2, 200)] + more, "int8" if block % 8 else "e4m3", "bf16", 4, 2, dim, page=page, block=block,
                 hnd=page % 16 == 0, seed=page).poison_unused()
        check_twice(c, f"page {page} block {block}")


@pytest.mark.parametrize("rows", [15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("dim", [64, 256])
def test_rows_around_a_tile(rows, dim):
    """Also around the count at which tiles of few rows give way to those of many."""
    for more in ([], [(1, 90)], [(0, 4)] * 300):
        c = Case([(rows, rows + 77)] + more, "int8", "f16", 1, 1, dim, seed=rows).poison_unused()
        check_twice(c, f"{rows} rows")


@pytest.mark.parametrize("keys", [1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 127, 128, 129, 192, 193])
def test_keys_around_a_block(keys):
    for dim in (128, 256):
        for new in (1, min(keys, 20)):
            c = Case([(new, keys)], "e4m3", "bf16", 32, 1, dim, seed=keys).poison_unused()
            check_twice(c, f"{keys} keys, {new} new")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 70), (63, 0), (64, 3), (65, 64), (129, 65), (1000, 4)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_over_cut_tiles(window, sinks, dim):
    for more in ([], [(0, 3)] * 60):
        c = Case([(50, 1500), (3, 900), (1, 2000)] + more, "int8", "bf16", 8, 2, dim, seed=window).poison_unused()
        c.window, c.sinks = window, sinks
        check_twice(c, f"{window}/{sinks}")


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-42])
def test_scales_of_chunks(scale):
    for lens in ([(40, 300)], [(1, 300), (2, 33)]):
        c = Case(lens, "int8", "f16", 2, 1, 64, seed=2).poison_unused()
        c.scale = scale
        c.check(c.run(), f"scale {scale}")


@pytest.mark.parametrize("code,dtype", KINDS)
def test_blocks_of_very_different_scales(code, dtype):
    """k and v of blocks whose scales are up to 2^30 apart (2^20 for binary16), small and large beside one another."""
    far = 30 if dtype == "bf16" else 10
    for lens in ([(1, 500), (1, 90)], [(40, 500), (1, 90)]):
        for dim in (64, 128):
            c = Case(lens, code, dtype, 4, 2, dim, block=8, seed=4)
            g = torch.Generator(device="cuda").manual_seed(9)
            shift = torch.randint(-far, far + 1, c.c.vs.shape, generator=g, device="cuda", dtype=I32)
            c.c.vs.copy_((c.c.vs.int() + shift).clamp(1, 130 if dtype == "f16" else 254).byte())
            c.c.ks.copy_((c.c.ks.int() + shift.flip(0) // 6).byte())
            c.check(c.run(), f"{code} {dtype} {dim}")
            c.check(c.run(torch.float32), f"{code} {dtype} {dim} float32")


def test_rising_maxima_of_chunks():
    """Scores that rise along the keys by far more than the slack of the running maximum, and fall again."""
    for dtype in ("f16", "bf16"):
        for lens in ([(40, 640)], [(1, 640)]):
            c = Case(lens, "int8", dtype, 2, 1, 64, block=8, seed=9)
            c.q[..., 0] = 8.0
            for j in range(640):
                at = c.table[0][j // 16], j % 16
                c.c.k[at[0], at[1], 0, 0] = (j if j < 400 else 800 - j) // 4
                c.c.ks[at[0], at[1] // 8] = 126
            c.check(c.run(), dtype)


def test_many_requests_of_both_kinds():
    """More requests than a workgroup has threads, rows few and many, by either kind of tile."""
    for choice in ([0, 1, 1, 1, 2, 30], [0, 0, 1, 1, 1, 1, 2]):
        rng = random.Random(11)
        lens = [(rng.choice(choice), rng.randrange(0, 120)) for _ in range(700)]
        check_twice(Case(lens, "e4m3", "f16", 2, 1, 64), "700 requests")


@pytest.mark.parametrize("dim", [64, 128])
def test_cut_tiles_past_the_first_requests(dim):
    """300 requests, short but for the last: few rows and many over thousands of keys, cut and joined."""
    for first in (1, 5):
        lens = [(first, 5 + r % 5) for r in range(295)] + [(1, 6000), (0, 9), (40, 3000), (5, 2500), (1, 4001)]
        check_twice(Case(lens, "int8", "f16", 4, 2, dim, seed=8), "the last of 300 requests")


# ------------------------------------------------------------------ tiles of several heads

@pytest.mark.parametrize("hq,hkv,dim,requests,keys,window", [
    (8, 8, 64, 64, 2600, 0), (16, 8, 128, 64, 2600, 0), (4, 2, 64, 128, 4200, 0), (6, 6, 128, 64, 3100, 0), (8, 8, 64, 70, 9000, 2400)])
def test_tiles_of_several_heads(hq, hkv, dim, requests, keys, window):
    """Many long requests: two or four heads to a tile, whole and cut, against the definition for some of them."""
    rng = random.Random(keys)
    lens = [(1, rng.randrange(keys // 2, 3 * keys // 2)) for _ in range(requests)]
    c = Case(lens, "e4m3" if dim == 64 else "int8", "bf16", hq, hkv, dim, seed=2)
    c.window, c.sinks = window, 5
    out = c.run()
    assert c.run().equal(out) and not c.work[:COUNTERS].any()
    some = [0, 1, requests // 2, requests - 1]
    y, bound, _ = ref.attn(c.q[some], c.c.k, c.c.ks, c.c.v, c.c.vs, ints([c.table[r] for r in some], "cpu"), ints(range(len(some) + 1), "cpu"),
                           ints([c.lens[r] for r in some], "cpu"), c.scale, window, 5, torch.bfloat16)
    assert ((out[some].double().cpu() - y).abs() <= bound).all()
    same_by_single_heads(c)


def same_by_single_heads(c):
    """The float32 result over the same values with a page's rows of one head together, which are read head by head: both
    within the weights' two pieces (2^-16), the scores' error (below 2^-14 for sums of 128 products of size 1) and the
    sums' rounding of the exact result, relative to the largest |v|."""
    a = c.run(torch.float32)
    k, v = c.c.k, c.c.v
    turned = lambda t: t.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(t.dtype)  # noqa: E731
    c.c.k, c.c.v = turned(k), turned(v)
    b = c.run(torch.float32)
    c.c.k, c.c.v = k, v
    largest = float(ref.values(v, c.c.vs).abs().max())
    assert float((a - b).abs().max()) <= 2 * (2.0 ** -16 + 2.0 ** -13 + 9000 / 8 * 2.0 ** -24) * largest


@pytest.mark.parametrize("hq,hkv,dim,requests,keys,new", [(32, 4, 64, 130, 2200, 1), (64, 4, 64, 130, 2200, 1), (8, 4, 128, 130, 2100, 5),
                                                        (24, 2, 128, 130, 4300, 3)])
def test_tiles_of_several_heads_and_many_rows(hq, hkv, dim, requests, keys, new):
    """Rows of all heads of a tile that are more than the 16 which are joined at a time, and several tiles a head."""
    rng = random.Random(hq)
    lens = [(rng.randrange(1, new + 1) if new > 1 else 1, rng.randrange(keys // 2, 3 * keys // 2)) for _ in range(requests)]
    c = Case(lens, "int8", "bf16", hq, hkv, dim, seed=3)
    out = c.run()
    assert c.run().equal(out) and not c.work[:COUNTERS].any()
    same_by_single_heads(c)


# ------------------------------------------------------------------ workspaces, plans, strides

def test_less_room_for_parts():
    """Room for some parts but not all, for the counters alone, and for nothing: tiles go whole."""
    c = Case([(40, 2000), (1, 3000)], "e4m3", "bf16", 4, 2, 128, seed=3)
    c.check(c.run(), "all")
    for size in (COUNTERS + 4 * 128 * 132 * 4, COUNTERS, 16):
        work = torch.zeros(size, dtype=torch.uint8, device="cuda")
        c.check(c.run(workspace=work), f"{size} bytes")
        assert not work[:COUNTERS].any()
    c.check(c.run(workspace=None), "none")


def test_one_workspace_for_many_shapes():
    """Counters and parts serve calls of any shapes after one another, without clearing."""
    work = paged.attn_workspace(256)
    for dim, lens in ((64, [(1, 3000)]), (256, [(30, 900)]), (128, [(1, 2000), (20, 700)]), (64, [(100, 1000)])):
        c = Case(lens, "int8", "bf16", 4, 1, dim, seed=dim)
        c.work = work
        check_twice(c, f"{dim} {lens}")


@pytest.mark.parametrize("lens", [[(60, 3000), (1, 5000)], [(1, 1), (70, 70)], [(1, 2500), (1, 70)]])
@pytest.mark.parametrize("window", [0, 700])
def test_tables_far_wider_than_the_keys(lens, window):
    """2^31 keys fit the table: the plan counts more than one block as one, and the last keys have no place."""
    c = Case(lens, "int8", "bf16", 16, 8, 64, page=128, seed=7).poison_unused()
    c.window, c.sinks = window, 4
    y, bound, mine = c.want(torch.bfloat16)
    assert mine.all()
    table = torch.full((len(lens), 1 << 24), -1, dtype=I32, device="cuda")
    table[:, :len(c.table[0])] = ints(c.table)
    first = None
    for _ in range(2):
        out = torch.full_like(c.q, 7.0)
        paged8.gemv_paged8_attn(c.q, *c.c.all, table, ints(c.starts), ints(c.lens), c.scale, out, c.work, window=window, sinks=4)
        assert ((out.double().cpu() - y).abs() <= bound).all()
        assert first is None or out.equal(first), "another result the second time"
        first = out
        assert not c.work[:COUNTERS].any()


@pytest.mark.parametrize("step", [1 << 26, 1 << 27])
def test_tokens_far_apart(step):
    """Pages of 16 whose tokens are 2^26 and 2^27 bytes apart, their scales as far: appended, read and attended to."""
    c = Case([(20, 100), (1, 60)], "int8", "bf16", 4, 2, 64, block=4, seed=9)
    shape, far = c.c.k.shape, (2 * 64, step, 64, 1)
    sshape, sfar = c.c.ks.shape, (2, step, 1)
    span = lambda n, s: sum((a - 1) * b for a, b in zip(n, s)) + 1  # noqa: E731
    k, v = (torch.empty(span(shape, far), device="cuda", dtype=torch.int8).as_strided(shape, far) for _ in "kv")
    ks, vs = (torch.empty(span(sshape, sfar), device="cuda", dtype=torch.uint8).as_strided(sshape, sfar) for _ in "kv")
    k.copy_(c.c.k), v.copy_(c.c.v), ks.copy_(c.c.ks), vs.copy_(c.c.vs)
    c.c.k, c.c.v, c.c.ks, c.c.vs = k, v, ks, vs
    run_append(c.c, "f32", "bf16", places(random.Random(3), [(3, 20), (6, 1)], 16, shape[0]), 2, 64)
    out = c.run()
    slots = torch.arange(shape[0] * 16, device="cuda", dtype=I32)
    back = torch.empty(shape[0] * 16, 2, 64, device="cuda")
    paged8.gemv_paged8_read(k, v, ks, vs, slots, back)
    c.c.k, c.c.v, c.c.ks, c.c.vs = (t.contiguous() for t in (k, v, ks, vs))
    assert back.double().cpu().equal(ref.values(c.c.k, c.c.ks).flatten(0, 1))
    c.check(out, "far")


# ------------------------------------------------------------------ the binding

def attn_of(c, out, **more):
    paged8.gemv_paged8_attn(c.q, *c.c.all, ints(c.table), ints(c.starts), ints(c.lens), 0.125, out, c.work, **more)


def test_calls_without_the_module(monkeypatch):
    """Every operator by the checks in Python alone: the same results."""
    c = Case([(1, 300), (9, 70)], "int8", "bf16")
    want, back = c.run(), torch.empty(30, 2, 64, device="cuda")
    slots = ints(range(-2, 28))
    paged8.gemv_paged8_read(*c.c.all, slots, back)
    monkeypatch.setitem(sys.modules, package.__name__ + "._paged_fast", None)
    monkeypatch.delattr(package, "_paged_fast", raising=False)
    for module in (paged, paged8):
        for name in ("_LIB", "_FAST", "_DEVICE"):
            monkeypatch.setattr(module, name, None)
    paged8.load()
    assert paged8._FAST is None
    assert c.run().equal(want)
    again, other = torch.empty_like(back), torch.empty_like(back)
    paged8.gemv_paged8_read(*c.c.all, slots, again, other)
    assert again.equal(back) and not other.equal(back)
    run_append(Cache("int8", 20, 16, 16, 2, 128), "f32", "bf16", [3, 4, 5, 20, 37], 8, 128)
    with pytest.raises(TypeError):
        paged8.gemv_paged8_attn(c.q.float(), *c.c.all, c.tt, c.qs, c.kl, 0.125, torch.empty_like(c.q), c.work)


def test_unusual_arguments_take_the_other_way():
    """What the C++ module does not take at once gives the same result through the checks in Python."""
    c = Case([(3, 40)], "e4m3", "f16", 2, 1, 64)
    want = c.run()
    got = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    attn_of(c, got, stream=side.cuda_stream)
    side.synchronize()
    assert got.equal(want)
    k, v, ks, vs = c.c.all
    got.zero_()
    paged8.gemv_paged8_attn(c.q, k, v, ks.view(torch.float8_e8m0fnu), vs.view(torch.float8_e8m0fnu), ints(c.table), ints(c.starts),
                            ints(c.lens), 0.125, got, c.work)
    assert got.equal(want)
    x = torch.randn(4, 1, 64, device="cuda")
    outs = []
    for positions, style in ((ints([0, 1, 2, 3]), 1), (ints([[0, 1, 2, 3]]), "pairs")):
        cache = paged8.cache(1, 4, 1, 64, "int8")
        out = torch.empty(4, 1, 64, device="cuda", dtype=torch.float16)
        paged8.gemv_paged8_append(x, x, x, positions, torch.ones(32, device="cuda"), ints([3, 2, 1, 0]), out, *cache, style=style)
        outs.append((out, *cache))
    assert all(a.equal(b) for a, b in zip(*outs))


def test_wrong_tensors_are_refused():
    c = Case([(3, 40)], "int8", "f16", 2, 1, 64)
    t, s, n = ints(c.table), ints(c.starts), ints(c.lens)
    out = torch.full_like(c.q, 7.0)

    def attn(q=c.q, k=c.c.k, v=c.c.v, ks=c.c.ks, vs=c.c.vs, t=t, s=s, n=n, out=out, work=c.work, **more):
        paged8.gemv_paged8_attn(q, k, v, ks, vs, t, s, n, 0.125, out, work, **more)

    for bad, error in ((dict(q=c.q.float()), TypeError), (dict(q=c.q.cpu()), TypeError), (dict(k=c.c.k[:1]), ValueError),
                       (dict(v=c.c.v.view(torch.float8_e4m3fn)), TypeError), (dict(ks=c.c.ks[:1]), ValueError), (dict(vs=c.c.vs.cpu()), TypeError),
                       (dict(ks=c.c.ks.int(), vs=c.c.vs.int()), TypeError), (dict(t=t.long()), TypeError), (dict(s=s[:1]), ValueError),
                       (dict(n=n.cpu()), TypeError), (dict(out=out[:2]), TypeError), (dict(out=out.double()), TypeError),
                       (dict(work=c.work[::2]), TypeError), (dict(t=t[0]), ValueError)):
        with pytest.raises(error):
            attn(**bad)
    for bad, status in ((dict(window=-1), "GEMV_E_DIM"), (dict(out=c.q), "GEMV_E_ALIAS"), (dict(out=out.bfloat16()), "GEMV_E_FMT"),
                        (dict(work=c.c.k.view(-1)), "GEMV_E_ALIAS"), (dict(work=c.c.ks.new_zeros(64)[8:]), "GEMV_E_ALIGN")):
        with pytest.raises(binding.GemvError, match=status):
            attn(**bad)
    x = torch.randn(3, 1, 64, device="cuda")
    q_out, none, i3 = torch.empty(3, 1, 64, device="cuda", dtype=torch.float16), torch.ones(32, device="cuda"), ints([0, 1, 2])
    for bad, error, match in ((dict(positions=ints([0, 1])), ValueError, "shape"), (dict(style="thirds"), KeyError, None),
                              (dict(q_out=q_out.float()), TypeError, "float16 or bfloat16"), (dict(slots=i3.long()), TypeError, "int32"),
                              (dict(k=x.half()), TypeError, "must be")):
        a = {**dict(q=x, k=x, v=x, positions=i3, inv_freq=none, slots=i3, q_out=q_out, style="halves"), **bad}
        with pytest.raises(error, match=match):
            paged8.gemv_paged8_append(a["q"], a["k"], a["v"], a["positions"], a["inv_freq"], a["slots"], a["q_out"], *c.c.all, style=a["style"])
    with pytest.raises(ValueError, match="has to be given"):
        paged8.gemv_paged8_read(*c.c.all, i3)
    with pytest.raises(ValueError, match="shape"):
        paged8.gemv_paged8_read(*c.c.all, i3, x[:2])
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        paged8.gemv_paged8_read(*c.c.all, i3, x.double())
    with pytest.raises(TypeError, match="must be"):
        paged8.gemv_paged8_read(*c.c.all, i3, x, x.half())
    with pytest.raises(binding.GemvError, match="GEMV_E_ALIAS"):
        paged8.gemv_paged8_read(*c.c.all, i3, x, x)
    torch.cuda.synchronize()
    assert (out == 7.0).all()


@pytest.mark.parametrize("code", ref.CODES)
def test_append_slot_many_times(code):
    """A slot many times over with values that grow: its block's other new tokens keep theirs."""
    n = 300
    c = Cache(code, 4, 16, 16, 2, 64, seed=1)
    before = c.copy()
    x = torch.randn(n, 2, 64, device="cuda") * torch.exp2(torch.arange(n, device="cuda") / 32.0)[:, None, None]
    slots = [21, 22, 23] + [25] * (n - 3)
    out = torch.empty(n, 2, 64, device="cuda", dtype=torch.bfloat16)
    paged8.gemv_paged8_append(x, x, x, ints([0] * n), torch.empty(0, device="cuda"), ints(slots), out, *c.all)
    for codes, byte, old, old_byte in ((c.k, c.ks, before[0], before[2]), (c.v, c.vs, before[1], before[3])):
        got, old = ref.values(codes, byte), ref.values(old, old_byte)
        step = ref.scales(byte.cpu())[1, 0][:, None]
        rest = [p for p in range(16) if p not in (5, 6, 7, 9)]
        for mine, want in ((got[1, 5:8], x[:3].double().cpu()), (got[1, rest], old[1, rest])):
            # each rounding, at scales that at least double: below a step of the last; for e4m3 2^-4 of the value at the
            # first and steps of 2^-9 after it
            tol = step if code == "int8" else 2.0 ** -4 * want.abs() + 2.0 ** -9 * step
            assert ((mine - want).abs() <= tol).all()


@pytest.mark.parametrize("lens", [[(40, 90), (1, 33)], [(1, 70), (1, 90)]])
def test_scales_of_a_page_far_apart(lens):
    """Neighbouring blocks' scales 300 million bytes apart: a page's sixteen span more than 32 bits."""
    c = Case(lens, "int8", "bf16", 2, 1, 64, block=1, seed=5)
    pages, step = c.c.ks.shape[0], 300_000_000
    room = torch.zeros(16 * step, dtype=torch.uint8, device="cuda")
    for i, name in enumerate(("ks", "vs")):
        far = room[i * pages:].as_strided((pages, 16, 1), (1, step, 1))
        far.copy_(getattr(c.c, name))
        setattr(c.c, name, far)
    c.check(c.run())


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("rot", [0, 50])
def test_append_large_block_in_any_order(code, rot):
    """Thousands of tokens of one block in no order, among places that hold others and are rescaled."""
    page = 4096
    c = Cache(code, 4, page, page, 1, 64, seed=6)
    slots = random.Random(3).sample(range(page + 1, 2 * page), 3000) + random.Random(4).sample(range(3 * page, 4 * page), 1000)
    run_append(c, "f32", "bf16", slots, 1, rot)


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("lens", [[(1, 70)], [(40, 90)]])
def test_scales_whose_product_passes_32_bits(code, lens):
    """Rows of q that are 0 weigh all keys alike, whatever the keys' scales and the softmax's."""
    c = Case(lens, code, "bf16", 2, 1, 64, seed=3)
    c.c.ks.fill_(240)
    c.q.zero_()
    c.scale = 2.0 ** 20
    c.check(c.run())
