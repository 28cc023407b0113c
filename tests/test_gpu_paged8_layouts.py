"""A cache in 8 bits whose pages carry their scales, in one buffer: every operator gives what it gives over four of
their own, and what lies between stays as it was."""
import random

import pytest
import torch

import paged8_ref as ref
from decode_gemv_elementwise_amd import paged8
from test_gpu_paged8 import I32, STEPS, Case, ints, places, run_append

pytestmark = pytest.mark.gpu

FILL = 77


def in_one(c):
    """The cache c's contents in one buffer: a page's k, 16 bytes, its v, its k scales, a byte, its v scales, room."""
    pages, page, heads, dim = c.k.shape
    codes, scales = page * heads * dim, c.ks.shape[1] * heads
    at = [0, codes + 16, 2 * codes + 16, 2 * codes + 17 + scales]
    step = -(-(at[3] + scales) // 16) * 16 + 32
    buffer = torch.full((pages, step), FILL, dtype=torch.uint8, device="cuda")
    parts = []
    for t, a in zip((c.k, c.v, c.ks, c.vs), at):
        n = codes if t.dim() == 4 else scales
        part = buffer[:, a:a + n].view(t.dtype).view(t.shape)
        part.copy_(t)
        parts.append(part)
    between = torch.ones(step, dtype=torch.bool, device="cuda")
    for a, n in zip(at, (codes, codes, scales, scales)):
        between[a:a + n] = False
    c.k, c.v, c.ks, c.vs = parts
    return buffer, between


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("block,dim", [(16, 64), (4, 128)])
def test_pages_that_carry_their_scales(code, block, dim):
    lens = [(20, 100), (1, 60), (3, 33)]
    c, other = (Case(lens, code, "bf16", 4, 2, dim, block=block, seed=9) for _ in "ab")
    buffer, between = in_one(c.c)
    for step in STEPS.values():
        slots = places(random.Random(3), [(p, n) for p, n in step if p + n < 60][:3], 16, c.c.k.shape[0])
        for one in (c, other):
            run_append(one.c, "f32", "bf16", slots, 4, dim)
    for a, b in zip(c.c.all, other.c.all):
        assert a.contiguous().view(torch.uint8).equal(b.contiguous().view(torch.uint8))
    slots = torch.arange(-1, c.c.k.shape[0] * 16 + 1, device="cuda", dtype=I32)
    backs = []
    for one in (c, other):
        k, v = (torch.empty(slots.numel(), 2, dim, device="cuda") for _ in "kv")
        paged8.gemv_paged8_read(*one.c.all, slots, k, v)
        backs.append((k, v))
    assert all(a.equal(b) for a, b in zip(*backs))
    assert c.run().equal(other.run())
    assert (buffer[:, between] == FILL).all()
