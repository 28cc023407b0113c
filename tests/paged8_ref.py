"""Plain 64-bit references of the operators over a paged cache in 8 bits, on the CPU,
from the definitions in include/gemv_paged8.h."""
import math

import torch

import paged_ref

MOST = {"int8": 127.0, "e4m3": 448.0}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
# half a step of a code relative to its size, and the smallest step's half beside it
HALF = {"int8": (0.0, 0.5), "e4m3": (2.0 ** -4, 2.0 ** -10)}


def code_of(t):
    return "int8" if t.dtype == torch.int8 else "e4m3"


def scales(bytes_):
    """2^(byte - 127) in 64 bits, NaN for 255."""
    b = bytes_.view(torch.uint8).double()
    return torch.where(b == 255, math.nan, torch.exp2(b - 127))


def values(codes, bytes_):
    """All values [pages, page, heads, dim] of a cache in 64 bits."""
    block = codes.shape[1] // bytes_.shape[1]
    return codes.cpu().float().double() * scales(bytes_.cpu()).repeat_interleave(block, 1)[..., None]


def rounded(x, code):
    """x rounded to the codes' numbers (ties to even), in 64 bits: whole ones, or 4 significant bits and steps of at
    least 2^-9."""
    if code == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def byte_for(amax, code):
    """The least byte from 1 up with amax <= MOST 2^(byte - 127); 255 for an infinity or NaN."""
    if not math.isfinite(amax):
        return 255
    b = 1
    while amax > MOST[code] * 2.0 ** (b - 127):
        b += 1
    return b


def attn(q, codes, bytes_k, codes_v, bytes_v, table, query_start, kv_len, scale, window, sinks, out_dtype):
    """paged_ref.attn over the values rounded to q's type."""
    k, v = values(codes, bytes_k).to(q.dtype), values(codes_v, bytes_v).to(q.dtype)
    return paged_ref.attn(q, k, v, table, query_start, kv_len, scale, window, sinks, out_dtype)
