"""The paged operators' checks on the host, with no GPU: the library exports
what include/gemv_paged.h declares, refuses every invalid argument with the
documented status before any launch, and the binding refuses tensors that a
launch would misread.  Addresses are plain integers; nothing dereferences them."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from decode_gemv_elementwise_amd import binding, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S = binding.STATUS_CODE
OK, NULL, DIM, FMT, ACT = 0, S["GEMV_E_NULL"], S["GEMV_E_DIM"], S["GEMV_E_FMT"], S["GEMV_E_ACT"]
LAYOUT, ALIAS, ALIGN = S["GEMV_E_LAYOUT"], S["GEMV_E_ALIAS"], S["GEMV_E_ALIGN"]
MB = 1 << 20
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    try:
        return paged.load()
    except ImportError as e:  # pragma: no cover - the build step makes it
        pytest.skip(str(e))


def test_library_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemv_paged.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gemv_paged_[a-z_]+)\s*\(", text))
    assert len(names) == 7
    for n in names:
        assert hasattr(lib, n), n


# ------------------------------------------------------------------ slots

SLOTS = dict(cached=1 * MB, fresh=2 * MB, requests=8, free=3 * MB, num_free=100, page=16, table=4 * MB, width=10, stride=12,
             tokens=40, start=5 * MB, kv=6 * MB, request=7 * MB, pos=8 * MB, slots=9 * MB, used=10 * MB)


def slots(**change):
    return paged.gemv_paged_slots_validate(*{**SLOTS, **change}.values())


def test_slots_accepts():
    assert slots() == OK
    assert slots(free=None, num_free=0) == OK
    assert slots(tokens=0, request=None, pos=None, slots=None) == OK
    assert slots(requests=1, stride=1) == OK
    assert slots(page=1) == OK and slots(page=65536) == OK
    assert slots(tokens=TOP, request=1 << 40, pos=2 << 40, slots=3 << 40) == OK


@pytest.mark.parametrize("change,want", [
    (dict(cached=None), NULL), (dict(fresh=None), NULL), (dict(free=None), NULL), (dict(table=None), NULL),
    (dict(start=None), NULL), (dict(kv=None), NULL), (dict(request=None), NULL), (dict(pos=None), NULL),
    (dict(slots=None), NULL), (dict(used=None), NULL),
    (dict(requests=0), DIM), (dict(requests=(1 << 20) + 1), DIM), (dict(num_free=-1), DIM), (dict(num_free=1 << 31), DIM),
    (dict(page=0), DIM), (dict(page=65537), DIM), (dict(width=0), DIM), (dict(width=1 << 31), DIM), (dict(tokens=-1), DIM),
    (dict(tokens=1 << 31), DIM), (dict(stride=9), LAYOUT), (dict(stride=1 << 31), LAYOUT), (dict(requests=1, stride=0), LAYOUT),
    (dict(cached=1 * MB + 2), ALIGN), (dict(slots=9 * MB + 1), ALIGN),
    (dict(table=1 * MB), ALIAS), (dict(start=2 * MB + 28), ALIAS), (dict(kv=3 * MB), ALIAS), (dict(used=4 * MB + 8), ALIAS),
    (dict(slots=8 * MB + 156), ALIAS), (dict(request=7 * MB, pos=7 * MB + 80), ALIAS), (dict(used=2 ** 64 - 4, kv=2 ** 64 - 8), ALIAS)])
def test_slots_refuses(change, want):
    assert slots(**change) == want


# ------------------------------------------------------------------ append

def cache(k=1 << 40, v=1 << 41, type=2, heads=8, dim=128, page=16, pages=64, ks=(16384, 1024, 128), vs=(16384, 1024, 128)):
    return paged.make_cache(k, v, type, heads, dim, page, pages, ks, vs)


APPEND = dict(q=16 * MB, k=32 * MB, v=48 * MB, src=0, tokens=100, q_heads=32, qs=4096, ks=1024, vs=1024, pos=64 * MB, axes=1,
              axis=None, inv=65 * MB, rot=128, style=0, slots=66 * MB, out=80 * MB)


def append(c=None, **change):
    return paged.gemv_paged_append_validate(*{**APPEND, **change}.values(), c or cache())


def test_append_accepts():
    assert append() == OK
    assert append(q=16 * MB, k=16 * MB + 16384, v=16 * MB + 20480, qs=6144, ks=6144, vs=6144) == OK
    assert append(rot=0, pos=None, inv=None) == OK
    assert append(axes=3, axis=67 * MB, style=1) == OK
    assert append(q=16 * MB + 4, src=0) == OK and append(q=16 * MB + 2, src=1) == OK
    assert append(tokens=0, q=None, k=None, v=None, pos=None, slots=None, out=None) == OK
    assert append(qs=0) == OK  # one row for all tokens
    assert append(cache(ks=(16384, 128, 2048), vs=(16384, 128, 2048))) == OK  # a page's rows of a head together
    assert append(cache(v=(1 << 40) + 2 * 16384, ks=(32768, 1024, 128), vs=(32768, 1024, 128))) == OK  # halves of a page
    assert append(cache(v=(1 << 40) + 256, ks=(32768, 2048, 256), vs=(32768, 2048, 256))) == OK  # k and v side by side


@pytest.mark.parametrize("change,want", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(pos=None), NULL), (dict(inv=None), NULL),
    (dict(slots=None), NULL), (dict(out=None), NULL), (dict(src=3), FMT), (dict(src=-1), FMT), (dict(style=2), ACT),
    (dict(style=-1), ACT), (dict(tokens=-1), DIM), (dict(tokens=1 << 31), DIM), (dict(q_heads=0), DIM),
    (dict(q_heads=4097), DIM), (dict(axes=0), DIM), (dict(axes=65), DIM), (dict(rot=-2), DIM), (dict(rot=130), DIM),
    (dict(rot=127), DIM), (dict(qs=-1), LAYOUT), (dict(ks=1 << 31), LAYOUT), (dict(vs=-8), LAYOUT), (dict(q=16 * MB + 2), ALIGN),
    (dict(src=2, k=32 * MB + 1), ALIGN), (dict(pos=64 * MB + 2), ALIGN), (dict(out=80 * MB + 8), ALIGN),
    (dict(out=16 * MB), ALIAS), (dict(out=48 * MB + 1024), ALIAS), (dict(out=1 << 40), ALIAS), (dict(slots=(1 << 41) + 64), ALIAS),
    (dict(pos=80 * MB), ALIAS), (dict(k=(1 << 40) + 4096), ALIAS), (dict(out=2 ** 64 - 16), ALIAS)])
def test_append_refuses(change, want):
    assert append(**change) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(type=0), FMT), (dict(type=3), FMT), (dict(heads=0), DIM),
    (dict(heads=4097), DIM), (dict(dim=0), DIM), (dict(dim=132), DIM), (dict(dim=520), DIM), (dict(page=0), DIM),
    (dict(page=65537), DIM), (dict(pages=0), DIM), (dict(pages=1 << 31), DIM), (dict(pages=1 << 28), DIM),
    (dict(ks=(16384, 1024, 0)), LAYOUT), (dict(ks=(16384, 1024, -128)), LAYOUT), (dict(ks=(16384, 1024, 132)), LAYOUT),
    (dict(ks=(1 << 31, 1024, 128)), LAYOUT), (dict(vs=(16384, 1024, 120)), LAYOUT), (dict(vs=(8192, 1024, 128)), LAYOUT),
    (dict(ks=(16384, 1016, 128)), LAYOUT), (dict(ks=(1024, 1024, 128)), LAYOUT), (dict(k=(1 << 40) + 8), ALIGN),
    (dict(v=(1 << 41) + 2), ALIGN), (dict(v=1 << 40), ALIAS), (dict(v=(1 << 40) + 16384), ALIAS),
    (dict(v=(1 << 40) + 16, ks=(32768, 2048, 256), vs=(32768, 2048, 256)), ALIAS),
    (dict(v=(1 << 40) + 256, ks=(32768, 2048, 256), vs=(32768, 2048, 128)), ALIAS)])
def test_cache_refuses(change, want):
    assert append(cache(**change)) == want


# ------------------------------------------------------------------ attention

ATTN = dict(q=16 * MB, qts=4096, qhs=128, c=None, table=32 * MB, width=40, stride=40, start=33 * MB, kv=34 * MB, requests=5,
            tokens=20, q_heads=32, scale=0.1, window=0, sinks=0, out=48 * MB, type=2, ots=4096, ohs=128, work=64 * MB,
            bytes=16 * MB)


def attn(**change):
    a = {**ATTN, **change}
    a["c"] = a["c"] or cache()
    return paged.gemv_paged_attn_validate(*a.values())


def test_attn_accepts():
    assert attn() == OK and attn(type=0) == OK and attn(work=None, bytes=0) == OK
    for dim in (64, 256):
        s = (16384 * dim // 128, 1024 * dim // 128, dim)
        assert attn(c=cache(dim=dim, ks=s, vs=s), qts=32 * dim, qhs=dim, ots=32 * dim, ohs=dim) == OK
    assert attn(tokens=0, q=None, out=None) == OK
    assert attn(window=TOP, sinks=TOP) == OK
    assert attn(ots=128, ohs=20 * 128) == OK  # heads outermost
    assert attn(c=cache(v=(1 << 40) + 256, ks=(32768, 2048, 256), vs=(32768, 2048, 256))) == OK


@pytest.mark.parametrize("change,want", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(start=None), NULL), (dict(kv=None), NULL),
    (dict(work=None), NULL), (dict(type=1), FMT), (dict(type=5), FMT), (dict(requests=0), DIM),
    (dict(requests=(1 << 20) + 1), DIM), (dict(tokens=-1), DIM), (dict(tokens=1 << 27), DIM), (dict(width=0), DIM),
    (dict(q_heads=0), DIM), (dict(q_heads=12), DIM), (dict(q_heads=4104), DIM), (dict(window=-1), DIM),
    (dict(window=1 << 31), DIM), (dict(sinks=-1), DIM), (dict(bytes=-1), DIM), (dict(scale=float("nan")), DIM),
    (dict(scale=float("inf")), DIM), (dict(stride=39), LAYOUT), (dict(qts=4100), LAYOUT), (dict(qhs=-128), LAYOUT),
    (dict(ots=4092), LAYOUT), (dict(ohs=64), LAYOUT), (dict(ots=0), LAYOUT), (dict(ots=2048), LAYOUT), (dict(ohs=1 << 31), LAYOUT),
    (dict(q=16 * MB + 8), ALIGN), (dict(out=48 * MB + 2), ALIGN), (dict(work=64 * MB + 4), ALIGN), (dict(table=32 * MB + 1), ALIGN),
    (dict(out=16 * MB), ALIAS), (dict(out=1 << 40), ALIAS), (dict(work=16 * MB), ALIAS), (dict(work=40 * MB, out=48 * MB), ALIAS),
    (dict(kv=48 * MB + 16), ALIAS), (dict(out=2 ** 64 - 4096), ALIAS), (dict(tokens=2 ** 25, ots=TOP // 8 * 8, type=0), ALIAS)])
def test_attn_refuses(change, want):
    assert attn(**change) == want


@pytest.mark.parametrize("dim", [8, 32, 96, 512])
def test_attn_refuses_other_dims(dim):
    s = (16 * 8 * dim, 8 * dim, dim)
    assert attn(c=cache(dim=dim, ks=s, vs=s)) == DIM


def test_attn_workspace():
    with pytest.raises(binding.GemvError, match="GEMV_E_DIM"):
        paged.gemv_paged_attn_workspace(96)
    sizes = [paged.gemv_paged_attn_workspace(d) for d in (64, 128, 256)]
    assert sizes == sorted(sizes) and all(s % 16 == 0 for s in sizes)


# ------------------------------------------------------------------ the binding

def _i(n):
    return torch.zeros(n, dtype=torch.int32)


def test_host_tensors_are_refused():
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="GPU"):
        paged.gemv_paged_slots(_i(2), _i(2), _i(4), 16, torch.zeros(2, 4, dtype=torch.int32), _i(3), _i(2), _i(3), _i(3), _i(3), _i(1))
    with pytest.raises(TypeError, match="GPU"):
        paged.gemv_paged_append(q, q[:, :2], q[:, :2], _i(3), torch.ones(32), _i(3), q, kc, kc.clone())
    with pytest.raises(TypeError, match="GPU"):
        paged.gemv_paged_attn(q, kc, kc, torch.zeros(1, 4, dtype=torch.int32), _i(2), _i(1), 0.125, q.clone())


def test_tensor_checks():
    """The checks that follow the device's, on host tensors through the helpers they share."""
    dev = torch.device("cpu")
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    paged._cache_of(kc, kc, dev)
    for bad in (kc.bfloat16(), kc[:3], kc[0], kc.transpose(2, 3)):
        with pytest.raises((TypeError, ValueError)):
            paged._cache_of(kc, bad, dev)
    with pytest.raises(TypeError):
        paged._cache_of(kc.int(), kc.int(), dev)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        paged._cache_of(kc.double(), kc.double(), dev)
    x = torch.zeros(3, 4, 64)
    assert paged._rows_of(x, "q", x.shape, torch.float32, dev)[1] == 256
    with pytest.raises(TypeError, match="lie together"):
        paged._rows_of(x.transpose(0, 1), "q", torch.Size((4, 3, 64)), torch.float32, dev)
    with pytest.raises(ValueError, match="shape"):
        paged._rows_of(x, "q", torch.Size((3, 5, 64)), torch.float32, dev)
    with pytest.raises(TypeError, match="must be"):
        paged._rows_of(x.half(), "q", x.shape, torch.float32, dev)
    t = torch.zeros(3, 8, dtype=torch.int32)
    assert paged._table_of(t[:, :4], 3, dev)[1:] == (4, 8)
    for bad in (t.long(), t[:2], t.t(), t[0]):
        with pytest.raises((TypeError, ValueError)):
            paged._table_of(bad, 3, dev)
    with pytest.raises(TypeError, match="contiguous"):
        paged._dense(torch.zeros(8, dtype=torch.int32)[::2], "slots", torch.int32)
    with pytest.raises(ValueError, match="shape"):
        paged._dense(_i(3), "slots", torch.int32, (4,))
    with pytest.raises(TypeError, match="int32"):
        paged._dense(torch.zeros(3), "slots", torch.int32)
