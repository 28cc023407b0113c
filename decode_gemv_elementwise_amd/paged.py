"""ctypes binding of ``include/gemv_paged.h``: the operators of a paged
key/value cache, in the same library as ``binding`` and by its rules.

Functions carry the C names.  Tensors are torch tensors on the current GPU;
every one is checked here (device, dtype, layout, size) before the library's
own checks, because the kernels get raw addresses.  The ``*_validate`` twins
run the library's host checks alone and take raw integer addresses too.
Launches go to ``stream`` (default: torch's current stream); as with any
launch outside torch, a tensor used on another stream than the one it was
made on has to be kept alive, or recorded on that stream, by the caller.

Calls go through ``_paged_fast`` first (C++, 1 us a call where the same checks
here take 6); what it does not take at once comes to the checks below, which
accept the call or raise.  Where that module is not built, or is another
interpreter's, every call goes through the checks here.

A cache is a pair of tensors ``[pages, page_size, heads, dim]`` of float16 or
bfloat16 with any strides whose innermost is 1 (a ``[pages, heads, page_size,
dim]`` buffer goes in as ``buffer.transpose(1, 2)``).
"""
import ctypes

from . import binding

TYPES = None  # torch dtype -> element type code, made on first use
STYLES = {"halves": 0, "pairs": 1}

_VP, _I64, _INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class GemvKvCache(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("type", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", _I64), ("k_stride", _I64 * 3), ("v_stride", _I64 * 3)]


_CACHEP = ctypes.POINTER(GemvKvCache)
_LIB = None
_FAST = None      # the module that checks and marshals a call's tensors at once, if it is built
_DEVICE = None    # () -> index of the current GPU, -1 if there is none or no module


def load():
    """The library, with the paged operators declared; torch's types are known after it."""
    global _LIB, _FAST, _DEVICE, TYPES
    if _LIB is not None:
        return _LIB
    import torch
    lib = binding.load()
    slots = [_VP, _VP, _I64, _VP, _I64, _I64, _VP, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP]
    append = [_VP, _VP, _VP, _INT, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _VP, _VP, _I64, _INT, _VP, _VP, _CACHEP]
    attn = [_VP, _I64, _I64, _CACHEP, _VP, _I64, _I64, _VP, _VP, _I64, _I64, _I64, ctypes.c_float, _I64, _I64, _VP,
            _INT, _I64, _I64, _VP, _I64]
    for name, args in (("gemv_paged_slots", slots), ("gemv_paged_append", append), ("gemv_paged_attn", attn)):
        getattr(lib, name).argtypes = args + [_VP]
        getattr(lib, name).restype = _INT
        getattr(lib, name + "_validate").argtypes = args
        getattr(lib, name + "_validate").restype = _INT
    lib.gemv_paged_attn_workspace.argtypes = [_I64]
    lib.gemv_paged_attn_workspace.restype = _I64
    TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    try:
        from . import _paged_fast
    except ImportError:
        _paged_fast = None
    _FAST, _DEVICE = _paged_fast, lambda: -1
    if _FAST is not None:
        _FAST.bind(*(ctypes.cast(getattr(lib, f), _VP).value
                     for f in ("gemv_paged_slots", "gemv_paged_append", "gemv_paged_attn")))
        if torch.cuda.is_available():
            _DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _LIB = lib
    return lib


def make_cache(k, v, type, heads, dim, page_size, num_pages, k_stride, v_stride) -> GemvKvCache:
    """A GemvKvCache from addresses and sizes (strides: page, token in page, head)."""
    return GemvKvCache(k, v, type, heads, dim, page_size, num_pages, (_I64 * 3)(*k_stride), (_I64 * 3)(*v_stride))


# ------------------------------------------------------------------ tensor checks

def _dense(t, name, dtype, shape=None, device=None):
    """Address of a contiguous tensor of this dtype (and shape), on the device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise TypeError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _device_of(t, name):
    """The device of the first tensor: the current GPU."""
    import torch
    if not t.is_cuda:
        raise TypeError(f"{name}: tensor arguments of a launching call must be on the GPU")
    if t.device.index != torch.cuda.current_device():
        raise TypeError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return t.device


def _cache_of(k_cache, v_cache, device):
    shape, ks, vs = k_cache.shape, k_cache.stride(), v_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must be [pages, page_size, heads, dim] alike, got {tuple(shape)} and "
                         f"{tuple(v_cache.shape)}")
    if max(shape[1:]) >= 2 ** 31:
        raise ValueError(f"page_size, heads and dim of a cache must be below 2^31, got {tuple(shape)}")
    if v_cache.dtype != k_cache.dtype or k_cache.dtype not in TYPES:
        raise TypeError(f"k_cache and v_cache must be float16 or bfloat16 alike, got {k_cache.dtype} and {v_cache.dtype}")
    if ks[3] != 1 or vs[3] != 1:
        raise TypeError("a cache's values of one head must lie together (innermost stride 1)")
    if k_cache.device != device or v_cache.device != device:
        raise TypeError(f"the caches are on {k_cache.device} and {v_cache.device}, expected {device}")
    return GemvKvCache(k_cache.data_ptr(), v_cache.data_ptr(), TYPES[k_cache.dtype], shape[2], shape[3], shape[1],
                       shape[0], ks[:3], vs[:3])


def _rows_of(t, name, shape, dtype, device):
    """Address and row stride of [tokens, heads, dim] whose heads lie together in a row."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    s = t.stride()
    if t.numel() and ((shape[2] > 1 and s[2] != 1) or (shape[1] > 1 and s[1] != shape[2])):
        raise TypeError(f"{name}: the heads of a token must lie together, one after the other")
    if t.device != device:
        raise TypeError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr(), s[0]


def _table_of(t, requests, device):
    import torch
    if t.dtype != torch.int32:
        raise TypeError(f"block_table must be torch.int32, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != requests:
        raise ValueError(f"block_table must be [{requests}, width], got {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise TypeError("a block_table row's entries must lie together")
    if t.device != device:
        raise TypeError(f"block_table is on {t.device}, expected {device}")
    return t.data_ptr(), t.shape[1], t.stride(0)


# ------------------------------------------------------------------ API (C names)

def gemv_paged_slots(cached, fresh, free_pages, page_size, block_table, query_start, kv_len, token_request, positions,
                     slots, used, stream=None):
    """Block tables and slot maps of a step from its requests' lengths: ``cached`` and ``fresh`` [requests] in;
    ``block_table`` [requests, width] extended by pages of ``free_pages``; ``query_start`` [requests + 1], ``kv_len``
    [requests], ``token_request``, ``positions`` and ``slots`` [tokens] and ``used`` [1] out, all int32."""
    lib = _LIB or load()
    device = _DEVICE()
    if device >= 0:
        st = _FAST.slots(cached, fresh, free_pages, page_size, block_table, query_start, kv_len, token_request, positions,
                         slots, used, device, binding._stream(stream))
        if st == 0:
            return
        if st is not None:
            binding._raise(st)
    import torch
    i32 = torch.int32
    dev = _device_of(cached, "cached")
    n, tokens = cached.numel(), slots.numel()
    table, width, stride = _table_of(block_table, n, dev)
    one, per = (n,), (tokens,)
    st = lib.gemv_paged_slots(
        _dense(cached, "cached", i32, one), _dense(fresh, "fresh", i32, one, dev), n,
        _dense(free_pages, "free_pages", i32, None, dev), free_pages.numel(), page_size, table, width, stride, tokens,
        _dense(query_start, "query_start", i32, (n + 1,), dev), _dense(kv_len, "kv_len", i32, one, dev),
        _dense(token_request, "token_request", i32, per, dev), _dense(positions, "positions", i32, per, dev),
        _dense(slots, "slots", i32, per, dev), _dense(used, "used", i32, (1,), dev), binding._stream(stream))
    if st != 0:
        binding._raise(st)


def gemv_paged_append(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, axis=None, style="halves",
                      stream=None):
    """Rotary positions for q [tokens, q_heads, dim] and k [tokens, heads, dim] (float32, float16 or bfloat16 rows, any
    row stride), q into ``q_out`` and k and v into the cache at ``slots`` [tokens].  ``positions`` is [tokens] or
    [axes, tokens] int32, ``inv_freq`` [rot / 2] float32, ``axis`` [rot / 2] int32 the axis of each pair."""
    lib = _LIB or load()
    device = _DEVICE()
    if device >= 0:
        st = _FAST.append(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, axis, STYLES.get(style, style),
                          device, binding._stream(stream))
        if st == 0:
            return
        if st is not None:
            binding._raise(st)
    import torch
    i32 = torch.int32
    dev = _device_of(q, "q")
    if q.dim() != 3 or q.dtype not in TYPES:
        raise TypeError(f"q must be [tokens, q_heads, dim] of float32, float16 or bfloat16, got {tuple(q.shape)} {q.dtype}")
    cache = _cache_of(k_cache, v_cache, dev)
    tokens, q_heads, dim = q.shape
    if dim != cache.dim:
        raise ValueError(f"q has heads of {dim} values, the cache of {cache.dim}")
    kv = (tokens, cache.heads, dim)
    qa, qs = _rows_of(q, "q", q.shape, q.dtype, dev)
    ka, ks = _rows_of(k, "k", kv, q.dtype, dev)
    va, vs = _rows_of(v, "v", kv, q.dtype, dev)
    axes = positions.shape[0] if positions.dim() == 2 else 1
    half = inv_freq.numel()
    st = lib.gemv_paged_append(
        qa, ka, va, TYPES[q.dtype], tokens, q_heads, qs, ks, vs,
        _dense(positions, "positions", i32, (axes, tokens) if positions.dim() == 2 else (tokens,), dev), axes,
        None if axis is None else _dense(axis, "axis", i32, (half,), dev),
        _dense(inv_freq, "inv_freq", torch.float32, (half,), dev), 2 * half,
        STYLES[style] if isinstance(style, str) else style, _dense(slots, "slots", i32, (tokens,), dev),
        _dense(q_out, "q_out", k_cache.dtype, (tokens, q_heads, dim), dev), cache, binding._stream(stream))
    if st != 0:
        binding._raise(st)


def gemv_paged_attn(q, k_cache, v_cache, block_table, query_start, kv_len, scale, dst, workspace=None, window=0, sinks=0,
                    stream=None):
    """Attention of every request's new tokens over its paged cache.  q [tokens, q_heads, dim] of the cache's type and
    dst alike (or float32), both with any token and head strides; ``block_table`` [requests, width], ``query_start``
    [requests + 1], ``kv_len`` [requests] int32; ``window`` > 0 limits a token to the last ``window`` keys and the first
    ``sinks``.  ``workspace`` (see ``attn_workspace``) lets the keys of few rows be split over the whole card."""
    lib = _LIB or load()
    device = _DEVICE()
    if device >= 0:
        st = _FAST.attn(q, k_cache, v_cache, block_table, query_start, kv_len, scale, dst, workspace, window, sinks, device,
                        binding._stream(stream))
        if st == 0:
            return
        if st is not None:
            binding._raise(st)
    import torch
    dev = _device_of(q, "q")
    cache = _cache_of(k_cache, v_cache, dev)
    if q.dim() != 3 or q.dtype != k_cache.dtype or q.shape[2] != cache.dim:
        raise TypeError(f"q must be [tokens, q_heads, {cache.dim}] of {k_cache.dtype}, got {tuple(q.shape)} {q.dtype}")
    if dst.shape != q.shape or dst.dtype not in TYPES:
        raise TypeError(f"dst must be {tuple(q.shape)} of the cache's type or float32, got {tuple(dst.shape)} {dst.dtype}")
    qs, os = q.stride(), dst.stride()
    if qs[2] != 1 or os[2] != 1:
        raise TypeError("the values of one head of q and dst must lie together (innermost stride 1)")
    if dst.device != dev:
        raise TypeError(f"dst is on {dst.device}, expected {dev}")
    requests = kv_len.numel()
    table, width, stride = _table_of(block_table, requests, dev)
    tokens, q_heads, _ = q.shape
    wa = wb = 0
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.device != dev:
            raise TypeError(f"workspace must be contiguous and on {dev}")
        wa, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.gemv_paged_attn(
        q.data_ptr(), qs[0], qs[1], cache, table, width, stride,
        _dense(query_start, "query_start", torch.int32, (requests + 1,), dev),
        _dense(kv_len, "kv_len", torch.int32, (requests,), dev), requests, tokens, q_heads, scale, window, sinks,
        dst.data_ptr(), TYPES[dst.dtype], os[0], os[1], wa, wb, binding._stream(stream))
    if st != 0:
        binding._raise(st)


def gemv_paged_attn_workspace(dim) -> int:
    """Bytes of the workspace that is enough for any gemv_paged_attn with heads of ``dim`` values."""
    n = load().gemv_paged_attn_workspace(dim)
    if n < 0:
        binding._raise(int(n))
    return n


def attn_workspace(dim, device="cuda"):
    """A workspace for gemv_paged_attn, zero as its first use wants it; one per stream, kept for the program's life."""
    import torch
    return torch.zeros(gemv_paged_attn_workspace(dim), dtype=torch.uint8, device=device)


def gemv_paged_slots_validate(*args) -> int:
    """The host checks of the C function, on its arguments (addresses as integers); no HIP call."""
    return load().gemv_paged_slots_validate(*args)


def gemv_paged_append_validate(*args) -> int:
    return load().gemv_paged_append_validate(*args)


def gemv_paged_attn_validate(*args) -> int:
    return load().gemv_paged_attn_validate(*args)
