"""The paged attention's tiles of many rows, shares that cut tiles, and the calls'
two ways through the binding, against the 64-bit references of paged_ref."""
import random

import pytest
import torch

import paged_ref
from decode_gemv_elementwise_amd import binding, paged
from test_gpu_paged import Case, I32, ints, run_append

pytestmark = pytest.mark.gpu

COUNTERS = 8192  # bytes at the workspace's start


def check_twice(c, what):
    """Right, the same bits again, and the counters as they were."""
    out = c.run()
    c.check(out, what)
    assert c.run().equal(out), f"{what}: another result the second time"
    assert not c.work[:COUNTERS].any(), f"{what}: counters left"
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(9, 5000)], [(40, 3000)], [(17, 4097), (1, 3000), (130, 1500)], [(33, 2000)] * 3])
def test_cut_tiles(lens, dim, dtype):
    """Few tiles over many keys: every tile is cut over many workgroups and joined."""
    c = Case(lens, dtype, 4, 2, dim, seed=dim).poison_unused()
    check_twice(c, f"{lens} {dim}")
    c.check(c.run(torch.float32), "float32")


@pytest.mark.parametrize("page", [1, 8, 12, 16, 24, 48, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_of_long_chunks(page, dim):
    """The three ways to bring a block: runs of 16 keys in one page, of 8, and any."""
    c = Case([(20, 700), (70, 333), (2, 200)], "bf16", 4, 2, dim, page=page, hnd=page % 16 == 0, seed=page).poison_unused()
    check_twice(c, f"page {page}")


@pytest.mark.parametrize("rows", [16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("dim", [64, 256])
def test_rows_around_a_tile(rows, dim):
    c = Case([(rows, rows + 77), (1, 90)], "f16", 1, 1, dim, seed=rows).poison_unused()
    check_twice(c, f"{rows} rows")


@pytest.mark.parametrize("keys", [1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 127, 128, 129, 192, 193])
def test_keys_around_a_block(keys):
    for dim in (128, 256):
        c = Case([(min(keys, 20), keys)], "bf16", 32, 1, dim, seed=keys).poison_unused()
        check_twice(c, f"{keys} keys")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 70), (63, 0), (64, 3), (65, 64), (129, 65), (1000, 4)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_over_cut_tiles(window, sinks, dim):
    c = Case([(50, 1500), (3, 900), (1, 2000)], "bf16", 8, 2, dim, seed=window).poison_unused()
    c.window, c.sinks = window, sinks
    check_twice(c, f"{window}/{sinks}")


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_special_values_in_long_rows(value):
    """In keys that all rows see, that some see, and behind the window."""
    for window in (0, 300):
        c = Case([(40, 1200), (20, 500)], "bf16", 2, 1, 64, seed=5)
        c.window, c.sinks = window, 3
        for r, j in ((0, 20), (0, 1175), (1, 470), (1, 1)):
            c.v[c.table[r][j // 16], j % 16, 0, 7 + j % 3] = value
        # weights this small against the row's sum are not held apart from 0: no key is far below the others
        c.q[:] = c.q * 0.05
        c.check(c.run(), f"{value} window {window}")


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-42])
def test_scales_of_chunks(scale):
    c = Case([(40, 300)], "f16", 2, 1, 64, seed=2).poison_unused()
    c.scale = scale
    c.check(c.run(), f"scale {scale}")


def test_rising_maxima_of_chunks():
    """Scores that rise along the keys by far more than the slack of the running maximum, and fall again."""
    for dtype in ("f16", "bf16"):
        c = Case([(40, 640)], dtype, 2, 1, 64, seed=9)
        c.q[..., 0] = 8.0
        for j in range(640):
            c.k[c.table[0][j // 16], j % 16, 0, 0] = (j if j < 400 else 800 - j) / 8.0
        c.check(c.run(), dtype)


def test_many_requests_of_both_kinds():
    """More requests than a workgroup has threads, rows few and many."""
    rng = random.Random(11)
    lens = [(rng.choice([0, 1, 1, 1, 2, 30]), rng.randrange(0, 120)) for _ in range(700)]
    check_twice(Case(lens, "f16", 2, 1, 64), "700 requests")


def test_less_room_for_parts():
    """Room for some parts but not all, for the counters alone, and for nothing: tiles go whole."""
    c = Case([(40, 2000), (1, 3000)], "bf16", 4, 2, 128, seed=3)
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
        c = Case(lens, "bf16", 4, 1, dim, seed=dim)
        c.work = work
        check_twice(c, f"{dim} {lens}")


def test_chunk_in_a_graph():
    """A chunk cut over workgroups, captured once and replayed for other values, eager work between."""
    c = Case([(40, 2000)], "bf16", 4, 2, 128)
    out = torch.empty_like(c.q)
    table, starts, lens = ints(c.table), ints(c.starts), ints(c.lens)

    def call(out):
        paged.gemv_paged_attn(c.q, c.k, c.v, table, starts, lens, c.scale, out, c.work)

    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for n in range(4):
        c.q.normal_()
        lens.fill_(2000 - 61 * n)
        c.lens = [2000 - 61 * n]
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(out)
        call(eager)
        torch.cuda.synchronize()
        assert out.equal(eager), f"replay {n}"
        c.check(out, f"replay {n}")


def test_more_tokens_than_a_grid_has_rows():
    """Rotary append past 2^16 tokens, wide rows and odd ones."""
    run_append("bf16", "bf16", 70001, 1, 1, 16, 16, 1, "halves", 64)
    run_append("f16", "f16", 65537, 1, 1, 8, 6, 1, "pairs", 64)


def test_far_pages_of_a_chunk():
    """A cache of more than 2^31 elements, its last pages used by a tile of many rows."""
    pages = 2 ** 31 // (16 * 8 * 128) + 40
    c = Case([(20, 300), (1, 60)], "bf16", 16, 8, 128)
    k, v = (torch.empty((pages, 16, 8, 128), device="cuda", dtype=torch.bfloat16) for _ in "kv")
    small = c.k.shape[0]
    k[-small:], v[-small:] = c.k, c.v
    y, bound, _ = paged_ref.attn(c.q, c.k, c.v, ints(c.table, "cpu"), ints(c.starts, "cpu"), ints(c.lens, "cpu"), c.scale,
                                 0, 0, torch.bfloat16)
    table = ints(c.table)
    table = torch.where(table >= 0, table + (pages - small), table)
    out = torch.empty_like(c.q)
    paged.gemv_paged_attn(c.q, k, v, table, ints(c.starts), ints(c.lens), c.scale, out, c.work)
    assert ((out.double().cpu() - y).abs() <= bound).all()


# ------------------------------------------------------------------ the binding

def test_unusual_arguments_take_the_other_way():
    """What the C++ module does not take at once gives the same result through the checks in Python."""
    c = Case([(3, 40)], "f16", 2, 1, 64)
    want = c.run()
    c.scale = int(1)
    one = c.run()
    c.scale = 1.0
    assert one.equal(c.run())
    got = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    paged.gemv_paged_attn(c.q, c.k, c.v, ints(c.table), ints(c.starts), ints(c.lens), 0.125, got, c.work, stream=side.cuda_stream)
    side.synchronize()
    assert got.equal(want)
    x = torch.randn(4, 1, 64, device="cuda")
    outs = []
    for positions in (ints([0, 1, 2, 3]), ints([[0, 1, 2, 3]])):
        kc, vc = (torch.zeros(1, 4, 1, 64, device="cuda", dtype=torch.float16) for _ in "kv")
        out = torch.empty(4, 1, 64, device="cuda", dtype=torch.float16)
        paged.gemv_paged_append(x, x, x, positions, torch.ones(32, device="cuda"), ints([3, 2, 1, 0]), out, kc, vc, style=1)
        outs.append((out, kc, vc))
    assert all(a.equal(b) for a, b in zip(*outs))


def test_wrong_tensors_are_refused():
    c = Case([(3, 40)], "f16", 2, 1, 64)
    t, s, n = ints(c.table), ints(c.starts), ints(c.lens)
    out = torch.full_like(c.q, 7.0)

    def attn(q=c.q, k=c.k, v=c.v, t=t, s=s, n=n, out=out, work=c.work, **more):
        paged.gemv_paged_attn(q, k, v, t, s, n, 0.125, out, work, **more)

    for bad, error in ((dict(q=c.q.float()), TypeError), (dict(q=c.q.cpu()), TypeError), (dict(k=c.k[:1]), ValueError),
                       (dict(v=c.v.bfloat16()), TypeError), (dict(t=t.long()), TypeError), (dict(s=s[:1]), ValueError),
                       (dict(n=n.cpu()), TypeError), (dict(out=out[:2]), TypeError), (dict(out=out.double()), TypeError),
                       (dict(work=c.work[::2]), TypeError), (dict(t=t[0]), ValueError)):
        with pytest.raises(error):
            attn(**bad)
    for bad, status in ((dict(window=-1), "GEMV_E_DIM"), (dict(out=c.q), "GEMV_E_ALIAS"),
                        (dict(work=c.k.view(-1)), "GEMV_E_ALIAS")):
        with pytest.raises(binding.GemvError, match=status):
            attn(**bad)
    x = torch.randn(3, 1, 64, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        paged.gemv_paged_append(x, x, x, ints([0, 1]), torch.ones(32, device="cuda"), ints([0, 1, 2]),
                                torch.empty(3, 1, 64, device="cuda", dtype=torch.float16), c.k, c.v)
    with pytest.raises(KeyError):
        paged.gemv_paged_append(x, x, x, ints([0, 1, 2]), torch.ones(32, device="cuda"), ints([0, 1, 2]),
                                torch.empty(3, 1, 64, device="cuda", dtype=torch.float16), c.k, c.v, style="thirds")
    one = torch.zeros(1, dtype=I32, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        paged.gemv_paged_slots(one, one, one, 16, t[:1], ints([0, 0, 0]), one.clone(), one.clone(), one.clone(), one.clone(),
                               one.clone())
    torch.cuda.synchronize()
    assert (out == 7.0).all()
