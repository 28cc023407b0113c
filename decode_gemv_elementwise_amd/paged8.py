"""ctypes binding of ``include/gemv_paged8.h``: the operators over a paged
key/value cache held in 8 bits, by the rules of ``paged`` (block tables and slot
maps are made by ``paged.gemv_paged_slots``; the attention's workspace by
``paged.attn_workspace``).

A cache is four tensors: the codes ``k_cache`` and ``v_cache`` ``[pages, page_size,
heads, dim]`` of int8 or float8_e4m3fn with any strides whose innermost is 1, and the
scales' bytes ``k_scale`` and ``v_scale`` ``[pages, page_size / block, heads]`` of uint8
(or float8_e8m0fnu) with any strides.  A value is its code times 2^(byte - 127).
``cache`` makes an empty one.
"""
import ctypes

from . import binding, paged
from .paged import STYLES, _dense, _device_of, _I64, _INT, _rows_of, _table_of, _VP

CODES = {"int8": 0, "e4m3": 1}


class GemvKvCache8(ctypes.Structure):
    _fields_ = [("k", _VP), ("v", _VP), ("k_scale", _VP), ("v_scale", _VP), ("code", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("block", ctypes.c_int32),
                ("num_pages", _I64), ("k_stride", _I64 * 3), ("v_stride", _I64 * 3), ("ks_stride", _I64 * 3),
                ("vs_stride", _I64 * 3)]


_CACHEP = ctypes.POINTER(GemvKvCache8)
_LIB = None
_FAST = None
_DEVICE = None


def load():
    """The library, with the operators over a cache in 8 bits declared."""
    global _LIB, _FAST, _DEVICE
    if _LIB is not None:
        return _LIB
    lib = paged.load()
    append = [_VP, _VP, _VP, _INT, _I64, _I64, _I64, _I64, _I64, _VP, _I64, _VP, _VP, _I64, _INT, _VP, _VP, _INT, _CACHEP]
    read = [_CACHEP, _VP, _I64, _VP, _VP, _INT, _I64, _I64]
    attn = [_VP, _INT, _I64, _I64, _CACHEP, _VP, _I64, _I64, _VP, _VP, _I64, _I64, _I64, ctypes.c_float, _I64, _I64, _VP,
            _INT, _I64, _I64, _VP, _I64]
    for name, args in (("gemv_paged8_append", append), ("gemv_paged8_read", read), ("gemv_paged8_attn", attn)):
        getattr(lib, name).argtypes = args + [_VP]
        getattr(lib, name).restype = _INT
        getattr(lib, name + "_validate").argtypes = args
        getattr(lib, name + "_validate").restype = _INT
    _FAST, _DEVICE = paged._FAST, paged._DEVICE
    if _FAST is not None:
        _FAST.bind8(*(ctypes.cast(getattr(lib, f), _VP).value
                      for f in ("gemv_paged8_append", "gemv_paged8_read", "gemv_paged8_attn")))
    _LIB = lib
    return lib


def make_cache(k, v, k_scale, v_scale, code, heads, dim, page_size, block, num_pages, k_stride, v_stride, ks_stride,
               vs_stride) -> GemvKvCache8:
    """A GemvKvCache8 from addresses and sizes (strides: page, token in page or block in page, head)."""
    return GemvKvCache8(k, v, k_scale, v_scale, code, heads, dim, page_size, block, num_pages, (_I64 * 3)(*k_stride),
                        (_I64 * 3)(*v_stride), (_I64 * 3)(*ks_stride), (_I64 * 3)(*vs_stride))


def cache(pages, page_size, heads, dim, code="e4m3", block=None, device="cuda"):
    """(k_cache, v_cache, k_scale, v_scale) of an empty cache; ``block`` tokens (default: a page) share a scale.  Blocks
    of more than 16 floor(1024 / dim) tokens (128 for heads of 128 values) are appended to many times slower."""
    import torch
    block = page_size if block is None else block
    if block < 1 or page_size % block:
        raise ValueError(f"block must divide page_size {page_size}, got {block}")
    dtype = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[code]
    codes = lambda: torch.zeros(pages, page_size, heads, dim, dtype=torch.int8, device=device).view(dtype)  # noqa: E731
    scales = lambda: torch.zeros(pages, page_size // block, heads, dtype=torch.uint8, device=device)  # noqa: E731
    return codes(), codes(), scales(), scales()


# ------------------------------------------------------------------ tensor checks

def _cache_of(k_cache, v_cache, k_scale, v_scale, device):
    import torch
    shape, ks, vs = k_cache.shape, k_cache.stride(), v_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must be [pages, page_size, heads, dim] alike, got {tuple(shape)} and "
                         f"{tuple(v_cache.shape)}")
    if max(shape[1:]) >= 2 ** 31:
        raise ValueError(f"page_size, heads and dim of a cache must be below 2^31, got {tuple(shape)}")
    code = {torch.int8: 0, torch.float8_e4m3fn: 1}.get(k_cache.dtype)
    if v_cache.dtype != k_cache.dtype or code is None:
        raise TypeError(f"k_cache and v_cache must be int8 or float8_e4m3fn alike, got {k_cache.dtype} and {v_cache.dtype}")
    if ks[3] != 1 or vs[3] != 1:
        raise TypeError("a cache's values of one head must lie together (innermost stride 1)")
    blocks = k_scale.shape[1] if k_scale.dim() == 3 else 0
    if k_scale.shape != v_scale.shape or k_scale.dim() != 3 or blocks < 1 or shape[1] % blocks or \
            k_scale.shape[0] != shape[0] or k_scale.shape[2] != shape[2]:
        raise ValueError(f"k_scale and v_scale must be [{shape[0]}, page_size / block, {shape[2]}] alike with block a divisor "
                         f"of {shape[1]}, got {tuple(k_scale.shape)} and {tuple(v_scale.shape)}")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.dtype not in (torch.uint8, torch.float8_e8m0fnu):
            raise TypeError(f"{name} must be uint8 or float8_e8m0fnu, got {t.dtype}")
    for t in (k_cache, v_cache, k_scale, v_scale):
        if t.device != device:
            raise TypeError(f"a part of the cache is on {t.device}, expected {device}")
    return make_cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), code, shape[2],
                      shape[3], shape[1], shape[1] // blocks, shape[0], ks[:3], vs[:3], k_scale.stride(), v_scale.stride())


# ------------------------------------------------------------------ API (C names)

def gemv_paged8_append(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, k_scale, v_scale, axis=None,
                       style="halves", stream=None):
    """Rotary positions for q and k as by ``paged.gemv_paged_append``, q into ``q_out`` (float16 or bfloat16), k and v
    quantised into the cache at ``slots`` [tokens]; tokens of one block are neighbours in the call."""
    lib = _LIB or load()
    device = _DEVICE()
    if device >= 0:
        st = _FAST.append8(q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, k_scale, v_scale, axis,
                           STYLES.get(style, style), device, binding._stream(stream))
        if st == 0:
            return
        if st is not None:
            binding._raise(st)
    import torch
    i32 = torch.int32
    dev = _device_of(q, "q")
    if q.dim() != 3 or q.dtype not in paged.TYPES:
        raise TypeError(f"q must be [tokens, q_heads, dim] of float32, float16 or bfloat16, got {tuple(q.shape)} {q.dtype}")
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    tokens, q_heads, dim = q.shape
    if dim != cache.dim:
        raise ValueError(f"q has heads of {dim} values, the cache of {cache.dim}")
    if q_out.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"q_out must be float16 or bfloat16, got {q_out.dtype}")
    kv = (tokens, cache.heads, dim)
    qa, qs = _rows_of(q, "q", q.shape, q.dtype, dev)
    ka, ks = _rows_of(k, "k", kv, q.dtype, dev)
    va, vs = _rows_of(v, "v", kv, q.dtype, dev)
    axes = positions.shape[0] if positions.dim() == 2 else 1
    half = inv_freq.numel()
    st = lib.gemv_paged8_append(
        qa, ka, va, paged.TYPES[q.dtype], tokens, q_heads, qs, ks, vs,
        _dense(positions, "positions", i32, (axes, tokens) if positions.dim() == 2 else (tokens,), dev), axes,
        None if axis is None else _dense(axis, "axis", i32, (half,), dev),
        _dense(inv_freq, "inv_freq", torch.float32, (half,), dev), 2 * half,
        STYLES[style] if isinstance(style, str) else style, _dense(slots, "slots", i32, (tokens,), dev),
        _dense(q_out, "q_out", q_out.dtype, (tokens, q_heads, dim), dev), paged.TYPES[q_out.dtype], cache,
        binding._stream(stream))
    if st != 0:
        binding._raise(st)


def gemv_paged8_read(k_cache, v_cache, k_scale, v_scale, slots, k_out=None, v_out=None, stream=None):
    """The values at ``slots`` [tokens] into ``k_out`` and ``v_out`` [tokens, heads, dim] of one type (float32, float16 or
    bfloat16, any row stride), zeros for a slot outside the cache.  Either may be None."""
    lib = _LIB or load()
    device = _DEVICE()
    if device >= 0:
        st = _FAST.read8(k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out, device, binding._stream(stream))
        if st == 0:
            return
        if st is not None:
            binding._raise(st)
    import torch
    dev = _device_of(k_cache, "k_cache")
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    tokens = slots.numel()
    out = k_out if k_out is not None else v_out
    if out is None:
        raise ValueError("k_out or v_out has to be given")
    if out.dtype not in paged.TYPES:
        raise TypeError(f"k_out and v_out must be float32, float16 or bfloat16, got {out.dtype}")
    rows = [(None, 0) if t is None else _rows_of(t, name, (tokens, cache.heads, cache.dim), out.dtype, dev)
            for t, name in ((k_out, "k_out"), (v_out, "v_out"))]
    st = lib.gemv_paged8_read(cache, _dense(slots, "slots", torch.int32, (tokens,), dev), tokens, rows[0][0], rows[1][0],
                              paged.TYPES[out.dtype], rows[0][1], rows[1][1], binding._stream(stream))
    if st != 0:
        binding._raise(st)


def gemv_paged8_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, query_start, kv_len, scale, dst, workspace=None,
                     window=0, sinks=0, stream=None):
    """``paged.gemv_paged_attn`` over a cache in 8 bits, whose values enter rounded to q's type (float16 or bfloat16);
    dst of q's type or float32."""
    lib = _LIB or load()
    device = _DEVICE()
    if device >= 0:
        st = _FAST.attn8(q, k_cache, v_cache, k_scale, v_scale, block_table, query_start, kv_len, scale, dst, workspace,
                         window, sinks, device, binding._stream(stream))
        if st == 0:
            return
        if st is not None:
            binding._raise(st)
    import torch
    dev = _device_of(q, "q")
    cache = _cache_of(k_cache, v_cache, k_scale, v_scale, dev)
    if q.dim() != 3 or q.dtype not in (torch.float16, torch.bfloat16) or q.shape[2] != cache.dim:
        raise TypeError(f"q must be [tokens, q_heads, {cache.dim}] of float16 or bfloat16, got {tuple(q.shape)} {q.dtype}")
    if dst.shape != q.shape or dst.dtype not in paged.TYPES:
        raise TypeError(f"dst must be {tuple(q.shape)} of q's type or float32, got {tuple(dst.shape)} {dst.dtype}")
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
    st = lib.gemv_paged8_attn(
        q.data_ptr(), paged.TYPES[q.dtype], qs[0], qs[1], cache, table, width, stride,
        _dense(query_start, "query_start", torch.int32, (requests + 1,), dev),
        _dense(kv_len, "kv_len", torch.int32, (requests,), dev), requests, tokens, q_heads, scale, window, sinks,
        dst.data_ptr(), paged.TYPES[dst.dtype], os[0], os[1], wa, wb, binding._stream(stream))
    if st != 0:
        binding._raise(st)


def gemv_paged8_append_validate(*args) -> int:
    """The host checks of the C function, on its arguments (addresses as integers); no HIP call."""
    return load().gemv_paged8_append_validate(*args)


def gemv_paged8_read_validate(*args) -> int:
    return load().gemv_paged8_read_validate(*args)


def gemv_paged8_attn_validate(*args) -> int:
    return load().gemv_paged8_attn_validate(*args)
