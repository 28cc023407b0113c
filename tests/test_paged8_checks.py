"""The checks of the operators over a paged cache in 8 bits on the host, with no GPU:
the library exports what include/gemv_paged8.h declares, refuses every invalid argument
with the documented status before any launch, and the binding refuses tensors that a
launch would misread.  Addresses are plain integers; nothing dereferences them."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from decode_gemv_elementwise_amd import binding, paged8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S = binding.STATUS_CODE
OK, NULL, DIM, FMT, ACT = 0, S["GEMV_E_NULL"], S["GEMV_E_DIM"], S["GEMV_E_FMT"], S["GEMV_E_ACT"]
LAYOUT, ALIAS, ALIGN = S["GEMV_E_LAYOUT"], S["GEMV_E_ALIAS"], S["GEMV_E_ALIGN"]
MB = 1 << 20
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    try:
        return paged8.load()
    except ImportError as e:  # pragma: no cover - the build step makes it
        pytest.skip(str(e))


def test_library_exports_every_declared_function(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemv_paged8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gemv_paged8_[a-z_]+)\s*\(", text))
    assert len(names) == 6
    for n in names:
        assert hasattr(lib, n), n


# ------------------------------------------------------------------ the cache and the append

def cache(k=1 << 40, v=1 << 41, k_scale=1 << 42, v_scale=1 << 43, code=0, heads=8, dim=128, page=16, block=16, pages=64,
          ks=(16384, 1024, 128), vs=(16384, 1024, 128), kss=(8, 8, 1), vss=(8, 8, 1)):
    return paged8.make_cache(k, v, k_scale, v_scale, code, heads, dim, page, block, pages, ks, vs, kss, vss)


APPEND = dict(q=16 * MB, k=32 * MB, v=48 * MB, src=0, tokens=100, q_heads=32, qs=4096, ks=1024, vs=1024, pos=64 * MB, axes=1,
              axis=None, inv=65 * MB, rot=128, style=0, slots=66 * MB, out=80 * MB, type=2)


def append(c=None, **change):
    return paged8.gemv_paged8_append_validate(*{**APPEND, **change}.values(), c or cache())


def test_append_accepts():
    assert append() == OK and append(type=1) == OK and append(cache(code=1)) == OK
    assert append(q=16 * MB, k=16 * MB + 16384, v=16 * MB + 20480, qs=6144, ks=6144, vs=6144) == OK
    assert append(rot=0, pos=None, inv=None) == OK
    assert append(axes=3, axis=67 * MB, style=1) == OK
    assert append(q=16 * MB + 4, src=0) == OK and append(q=16 * MB + 2, src=1) == OK
    assert append(tokens=0, q=None, k=None, v=None, pos=None, slots=None, out=None) == OK
    assert append(qs=0) == OK  # one row for all tokens
    assert append(cache(ks=(16384, 128, 2048), vs=(16384, 128, 2048))) == OK  # a page's rows of a head together
    assert append(cache(v=(1 << 40) + 16384, ks=(32768, 1024, 128), vs=(32768, 1024, 128))) == OK  # halves of a page
    assert append(cache(v=(1 << 40) + 128, ks=(32768, 2048, 256), vs=(32768, 2048, 256))) == OK  # k and v side by side
    assert append(cache(block=4, kss=(32, 8, 1), vss=(32, 1, 4))) == OK
    assert append(cache(block=1, kss=(128, 8, 1), vss=(TOP, 8, 1))) == OK
    assert append(cache(v_scale=(1 << 42) + 8, kss=(16, 8, 1), vss=(16, 8, 1))) == OK  # scales of k and v side by side
    assert append(cache(v_scale=(1 << 42) + 1, kss=(16, 16, 2), vss=(16, 16, 2))) == OK
    assert append(cache(page=65536, block=65536, pages=2, ks=(1 << 26, 1024, 128), vs=(1 << 26, 1024, 128))) == OK


@pytest.mark.parametrize("change,want", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(pos=None), NULL), (dict(inv=None), NULL),
    (dict(slots=None), NULL), (dict(out=None), NULL), (dict(src=3), FMT), (dict(src=-1), FMT), (dict(type=0), FMT),
    (dict(type=3), FMT), (dict(style=2), ACT), (dict(style=-1), ACT), (dict(tokens=-1), DIM), (dict(tokens=1 << 31), DIM), (dict(tokens=(1 << 30) + 1), DIM),
    (dict(q_heads=0), DIM), (dict(q_heads=4097), DIM), (dict(axes=0), DIM), (dict(axes=65), DIM), (dict(rot=-2), DIM),
    (dict(rot=130), DIM), (dict(rot=127), DIM), (dict(qs=-1), LAYOUT), (dict(ks=1 << 31), LAYOUT), (dict(vs=-8), LAYOUT),
    (dict(q=16 * MB + 2), ALIGN), (dict(src=2, k=32 * MB + 1), ALIGN), (dict(pos=64 * MB + 2), ALIGN), (dict(out=80 * MB + 8), ALIGN),
    (dict(out=16 * MB), ALIAS), (dict(out=48 * MB + 1024), ALIAS), (dict(out=1 << 40), ALIAS), (dict(slots=(1 << 41) + 64), ALIAS),
    (dict(pos=80 * MB), ALIAS), (dict(k=(1 << 40) + 4096), ALIAS), (dict(out=2 ** 64 - 16), ALIAS), (dict(out=1 << 42), ALIAS),
    (dict(slots=(1 << 43) + 8), ALIAS), (dict(inv=(1 << 42) + 500), ALIAS)])
def test_append_refuses(change, want):
    assert append(**change) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k_scale=None), NULL), (dict(v_scale=None), NULL), (dict(code=2), FMT),
    (dict(code=-1), FMT), (dict(heads=0), DIM), (dict(heads=4097), DIM), (dict(dim=0), DIM), (dict(dim=136), DIM), (dict(dim=528), DIM),
    (dict(page=0), DIM), (dict(page=65537), DIM), (dict(pages=0), DIM), (dict(pages=1 << 31), DIM), (dict(pages=1 << 28), DIM),
    (dict(block=0), DIM), (dict(block=-16), DIM), (dict(block=5), DIM), (dict(block=32), DIM),
    (dict(ks=(16384, 1024, 0)), LAYOUT), (dict(ks=(16384, 1024, -128)), LAYOUT), (dict(ks=(16384, 1024, 136)), LAYOUT),
    (dict(ks=(1 << 31, 1024, 128)), LAYOUT), (dict(vs=(16384, 1024, 112)), LAYOUT), (dict(vs=(8192, 1024, 128)), LAYOUT),
    (dict(ks=(16384, 1008, 128)), LAYOUT), (dict(ks=(1024, 1024, 128)), LAYOUT), (dict(kss=(8, 8, 0)), LAYOUT),
    (dict(kss=(7, 8, 1)), LAYOUT), (dict(vss=(8, 8, -1)), LAYOUT), (dict(vss=(1 << 31, 8, 1)), LAYOUT), (dict(block=4, kss=(16, 8, 1)), LAYOUT),
    (dict(k=(1 << 40) + 8), ALIGN), (dict(v=(1 << 41) + 2), ALIGN), (dict(v=1 << 40), ALIAS), (dict(v=(1 << 40) + 8192), ALIAS),
    (dict(v=(1 << 40) + 16, ks=(32768, 2048, 256), vs=(32768, 2048, 256)), ALIAS),
    (dict(v=(1 << 40) + 128, ks=(32768, 2048, 256), vs=(32768, 2048, 128)), ALIAS), (dict(k_scale=(1 << 40) + 5), ALIAS),
    (dict(v_scale=(1 << 40) + 5), ALIAS), (dict(k_scale=(1 << 41)), ALIAS), (dict(v_scale=1 << 42), ALIAS),
    (dict(v_scale=(1 << 42) + 4, kss=(16, 8, 1), vss=(16, 8, 1)), ALIAS), (dict(v_scale=2 ** 64 - 20), ALIAS)])
def test_cache_refuses(change, want):
    assert append(cache(**change)) == want


# ------------------------------------------------------------------ reading

READ = dict(slots=16 * MB, tokens=100, k=32 * MB, v=48 * MB, type=2, ks=1024, vs=1024)


def read(c=None, **change):
    return paged8.gemv_paged8_read_validate(c or cache(), *{**READ, **change}.values())


def test_read_accepts():
    assert read() == OK and read(type=0) == OK and read(type=1) == OK
    assert read(k=None) == OK and read(v=None) == OK and read(k=None, ks=-5) == OK
    assert read(tokens=0, slots=None, k=None, v=None) == OK
    assert read(ks=2048, v=32 * MB + 2048, vs=2048) == ALIAS  # rows of k and v side by side: spans meet
    assert read(tokens=1, ks=0, vs=3) == OK
    assert read(cache(v=1 << 40)) == OK  # nothing is written there


@pytest.mark.parametrize("change,want", [
    (dict(slots=None), NULL), (dict(k=None, v=None), NULL), (dict(type=3), FMT), (dict(type=-1), FMT), (dict(tokens=-1), DIM),
    (dict(tokens=1 << 31), DIM), (dict(ks=1028), LAYOUT), (dict(vs=1016), LAYOUT), (dict(ks=-1024), LAYOUT), (dict(vs=1 << 31), LAYOUT),
    (dict(slots=16 * MB + 2), ALIGN), (dict(k=32 * MB + 8), ALIGN), (dict(v=48 * MB + 4), ALIGN), (dict(v=32 * MB + 1024), ALIAS),
    (dict(k=1 << 40), ALIAS), (dict(v=(1 << 41) + 1024), ALIAS), (dict(k=16 * MB), ALIAS), (dict(k=(1 << 42) + 256), ALIAS),
    (dict(v=1 << 43), ALIAS), (dict(k=2 ** 64 - 16), ALIAS)])
def test_read_refuses(change, want):
    assert read(**change) == want


@pytest.mark.parametrize("change,want", [(dict(k_scale=None), NULL), (dict(block=3), DIM), (dict(kss=(8, 8, 0)), LAYOUT), (dict(k=(1 << 40) + 1), ALIGN)])
def test_read_and_attn_refuse_caches(change, want):
    assert read(cache(**change)) == want and attn(c=cache(**change)) == want


# ------------------------------------------------------------------ attention

ATTN = dict(q=16 * MB, qtype=2, qts=4096, qhs=128, c=None, table=32 * MB, width=40, stride=40, start=33 * MB, kv=34 * MB, requests=5,
            tokens=20, q_heads=32, scale=0.1, window=0, sinks=0, out=48 * MB, type=2, ots=4096, ohs=128, work=64 * MB,
            bytes=16 * MB)


def attn(**change):
    a = {**ATTN, **change}
    a["c"] = a["c"] or cache()
    return paged8.gemv_paged8_attn_validate(*a.values())


def test_attn_accepts():
    assert attn() == OK and attn(type=0) == OK and attn(work=None, bytes=0) == OK and attn(qtype=1, type=1) == OK
    for dim in (64, 256):
        s = (16384 * dim // 128, 1024 * dim // 128, dim)
        assert attn(c=cache(dim=dim, ks=s, vs=s), qts=32 * dim, qhs=dim, ots=32 * dim, ohs=dim) == OK
    assert attn(tokens=0, q=None, out=None) == OK
    assert attn(window=TOP, sinks=TOP) == OK
    assert attn(ots=128, ohs=20 * 128) == OK  # heads outermost
    assert attn(c=cache(v=(1 << 40) + 128, ks=(32768, 2048, 256), vs=(32768, 2048, 256))) == OK


@pytest.mark.parametrize("change,want", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(start=None), NULL), (dict(kv=None), NULL),
    (dict(work=None), NULL), (dict(type=1), FMT), (dict(type=5), FMT), (dict(qtype=0, type=0), FMT), (dict(qtype=1), FMT),
    (dict(requests=0), DIM), (dict(requests=(1 << 20) + 1), DIM), (dict(tokens=-1), DIM), (dict(tokens=1 << 27), DIM), (dict(width=0), DIM),
    (dict(q_heads=0), DIM), (dict(q_heads=12), DIM), (dict(q_heads=4104), DIM), (dict(window=-1), DIM),
    (dict(window=1 << 31), DIM), (dict(sinks=-1), DIM), (dict(bytes=-1), DIM), (dict(scale=float("nan")), DIM),
    (dict(scale=float("inf")), DIM), (dict(stride=39), LAYOUT), (dict(qts=4100), LAYOUT), (dict(qhs=-128), LAYOUT),
    (dict(ots=4092), LAYOUT), (dict(ohs=64), LAYOUT), (dict(ots=0), LAYOUT), (dict(ots=2048), LAYOUT), (dict(ohs=1 << 31), LAYOUT),
    (dict(q=16 * MB + 8), ALIGN), (dict(out=48 * MB + 2), ALIGN), (dict(work=64 * MB + 4), ALIGN), (dict(table=32 * MB + 1), ALIGN),
    (dict(out=16 * MB), ALIAS), (dict(out=1 << 40), ALIAS), (dict(out=1 << 42), ALIAS), (dict(work=16 * MB), ALIAS),
    (dict(work=40 * MB, out=48 * MB), ALIAS), (dict(kv=48 * MB + 16), ALIAS), (dict(out=2 ** 64 - 4096), ALIAS),
    (dict(tokens=2 ** 25, ots=TOP // 8 * 8, type=0), ALIAS)])
def test_attn_refuses(change, want):
    assert attn(**change) == want


@pytest.mark.parametrize("dim", [16, 32, 96, 512])
def test_attn_refuses_other_dims(dim):
    s = (16 * 8 * dim, 8 * dim, dim)
    assert attn(c=cache(dim=dim, ks=s, vs=s)) == DIM


# ------------------------------------------------------------------ the binding

def _i(n):
    return torch.zeros(n, dtype=torch.int32)


def test_empty_caches():
    k, v, ks, vs = paged8.cache(5, 32, 2, 64, "e4m3", block=8, device="cpu")
    assert k.shape == v.shape == (5, 32, 2, 64) and k.dtype == torch.float8_e4m3fn and ks.shape == vs.shape == (5, 4, 2)
    assert paged8.cache(5, 32, 2, 64, "int8", device="cpu")[2].shape == (5, 1, 2)
    for block in (0, 5, 64):
        with pytest.raises(ValueError, match="divide"):
            paged8.cache(5, 32, 2, 64, block=block, device="cpu")


def test_host_tensors_are_refused():
    c = paged8.cache(4, 16, 2, 64, "int8", device="cpu")
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="GPU"):
        paged8.gemv_paged8_append(q, q[:, :2], q[:, :2], _i(3), torch.ones(32), _i(3), q, *c)
    with pytest.raises(TypeError, match="GPU"):
        paged8.gemv_paged8_read(*c, _i(3), q[:, :2], q[:, 2:])
    with pytest.raises(TypeError, match="GPU"):
        paged8.gemv_paged8_attn(q, *c, torch.zeros(1, 4, dtype=torch.int32), _i(2), _i(1), 0.125, q.clone())


def test_tensor_checks():
    """The checks that follow the device's, on host tensors."""
    dev = torch.device("cpu")
    for code in ("int8", "e4m3"):
        k, v, ks, vs = paged8.cache(4, 16, 2, 64, code, block=4, device="cpu")
        c = paged8._cache_of(k, v, ks, vs, dev)
        assert (c.code, c.heads, c.dim, c.page_size, c.block, c.num_pages) == (paged8.CODES[code], 2, 64, 16, 4, 4)
        assert list(c.k_stride) == [2048, 128, 64] and list(c.ks_stride) == [8, 2, 1]
        paged8._cache_of(k, v, ks.view(torch.float8_e8m0fnu), vs, dev)
        other = torch.float8_e4m3fn if code == "int8" else torch.int8
        for bad in (v.view(other), v.view(torch.uint8), v[:3], v[0], v.transpose(2, 3), v.float()):
            with pytest.raises((TypeError, ValueError)):
                paged8._cache_of(k, bad, ks, vs, dev)
        for bad in (ks[:3], ks[:, :3], ks[0], ks[..., :1], ks.int(), ks.view(torch.int8), ks[:, :0]):
            with pytest.raises((TypeError, ValueError)):
                paged8._cache_of(k, v, bad, vs, dev)
            with pytest.raises((TypeError, ValueError)):
                paged8._cache_of(k, v, bad, bad, dev)
        with pytest.raises(TypeError, match="int8 or float8"):
            paged8._cache_of(k.view(torch.uint8), k.view(torch.uint8), ks, vs, dev)
        with pytest.raises(TypeError, match="expected"):
            paged8._cache_of(k, v, ks, vs, torch.device("meta"))


def test_cache_sizes_past_32_bits_are_refused():
    dev = torch.device("meta")
    for shape in ((1, 2 ** 32 + 16, 1, 16), (1, 16, 2 ** 32 + 1, 16), (1, 1, 1, 2 ** 32 + 64)):
        t = torch.empty(shape, dtype=torch.int8, device=dev)
        s = torch.empty((1, 1, shape[2]), dtype=torch.uint8, device=dev)
        with pytest.raises(ValueError, match="2\\^31"):
            paged8._cache_of(t, t, s, s, dev)
