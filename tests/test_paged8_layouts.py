"""Where a cache's codes and scales may lie in memory: the append takes what shares no byte, and refuses
what does.  Addresses are plain integers; nothing dereferences them."""
import itertools
import random

import pytest

pytest.importorskip("torch")

from decode_gemv_elementwise_amd import binding, paged8

OK, ALIAS = 0, binding.STATUS_CODE["GEMV_E_ALIAS"]
MB = 1 << 20
BASE = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    try:
        return paged8.load()
    except ImportError as e:  # pragma: no cover - the build step makes it
        pytest.skip(str(e))


def append(cache):
    heads, dim = cache.heads, cache.dim
    return paged8.gemv_paged8_append_validate(16 * MB, 32 * MB, 48 * MB, 0, 10, heads, heads * dim, heads * dim, heads * dim, 64 * MB, 1,
                                              None, 65 * MB, dim, 0, 66 * MB, 80 * MB, 2, cache)


def paged(k, v, ks, vs, step, heads=2, dim=64, page=16, block=4, pages=8, scale_step=None):
    """Offsets of the four within a page's `step` bytes, each of them in the order [token][head]."""
    code = (step, heads * dim, dim)
    scale = (scale_step or step, heads, 1)
    return paged8.make_cache(BASE + k, BASE + v, BASE + ks, BASE + vs, 1, heads, dim, page, block, pages, code, code, scale, scale)


CODES, SCALES = 2 * 64 * 16, 2 * 4  # bytes of a page's k and of its scales


@pytest.mark.parametrize("k,v,ks,vs,step", [
    (0, CODES, 2 * CODES, 2 * CODES + SCALES, 2 * CODES + 2 * SCALES),                   # k, v, their scales: 16 bytes of both
    (0, CODES + 16, CODES, CODES + 16 + CODES, 2 * CODES + 32),                          # each followed by its own
    (32, 32 + CODES, 0, 16, 2 * CODES + 32),                                             # scales first
    (0, CODES, 2 * CODES + 100, 2 * CODES + 3, 4 * CODES)])                              # room between and behind
def test_a_page_may_carry_its_scales(k, v, ks, vs, step):
    assert append(paged(k, v, ks, vs, step)) == OK
    assert append(paged(k, v, ks, vs, step, pages=1)) == OK


def test_scales_of_another_page_may_lie_there():
    """Scales that begin some pages behind their codes, or before them."""
    step = 2 * CODES + 2 * SCALES
    for pages in (-5, -1, 1, 3, 100):
        assert append(paged(0, CODES, 2 * CODES + pages * step, 2 * CODES + SCALES + pages * step, step)) == OK
        assert append(paged(0, CODES, 2 * CODES - 1 + pages * step, 2 * CODES + SCALES + pages * step, step)) == (OK if abs(pages) == 100 else ALIAS)


@pytest.mark.parametrize("ks,vs,step", [
    (2 * CODES - 1, 2 * CODES + SCALES, 2 * CODES + 2 * SCALES),          # a scale on v's last code
    (2 * CODES, 2 * CODES + SCALES - 1, 2 * CODES + 2 * SCALES),          # on the other scales
    (2 * CODES, 2 * CODES + SCALES + 1, 2 * CODES + 2 * SCALES),          # on the next page's first code
    (CODES, 2 * CODES, 2 * CODES + 2 * SCALES), (0, 2 * CODES, 2 * CODES + 2 * SCALES)])
def test_pages_whose_scales_meet_codes_are_refused(ks, vs, step):
    assert append(paged(0, CODES, ks, vs, step)) == ALIAS


def test_scales_of_other_page_strides_are_refused():
    step = 2 * CODES + 2 * SCALES
    assert append(paged(0, CODES, 2 * CODES, 2 * CODES + SCALES, step, scale_step=2 * step)) == ALIAS


def addresses(base, stride, extent, row):
    return {base + sum(i * s for i, s in zip(at, stride)) + e for at in itertools.product(*map(range, extent)) for e in range(row)}


def test_what_is_accepted_shares_no_byte():
    """Random places and orders in one buffer, counted byte by byte."""
    rng = random.Random(1)
    heads, dim, page, pages = 2, 16, 4, 3
    taken = refused = within = 0
    for _ in range(6000):
        block = rng.choice([1, 2, 4])
        blocks = page // block
        codes, scales = heads * dim * page, heads * blocks
        step = rng.choice([2 * codes + 16 * (-(-2 * scales // 16)), 2 * codes + 64, 4 * codes, codes])
        order = lambda n, row, whole: rng.choice([(whole, heads * row, row), (whole, row, n * row)])  # noqa: E731
        code, scale = order(page, dim, step), order(blocks, 1, rng.choice([step, step, step, scales, 2 * scales]))
        some = [0, codes, 2 * codes, 2 * codes + scales, codes + 16, step, 2 * codes + 32, 4 * codes, 100000]
        k, v = (16 * (rng.choice(some) // 16) for _ in "kv")
        ks, vs = (rng.choice(some) + rng.choice([0, 0, 0, -1, 1, scales, -scales, step]) for _ in "kv")
        c = paged8.make_cache(BASE + k, BASE + v, BASE + ks, BASE + vs, 0, heads, dim, page, block, pages, code, code, scale, scale)
        st = append(c)
        assert st in (OK, ALIAS, binding.STATUS_CODE["GEMV_E_LAYOUT"])
        refused += st != OK
        if st != OK:
            continue
        taken += 1
        parts = [addresses(k, code, (pages, page, heads), dim), addresses(v, code, (pages, page, heads), dim),
                 addresses(ks, scale, (pages, blocks, heads), 1), addresses(vs, scale, (pages, blocks, heads), 1)]
        assert all(a.isdisjoint(b) for a, b in itertools.combinations(parts, 2))
        spans = [(min(p), max(p)) for p in parts]
        within += any(a[0] <= b[1] and b[0] <= a[1] for a in spans[:2] for b in spans[2:])
    assert taken > 100 and refused > 100 and within > 30
