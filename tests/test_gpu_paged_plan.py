"""The paged attention's plan where its line is counted in coarse units, past the
first 256 requests, and over a cache whose tokens are far apart."""
import pytest
import torch

import paged_ref
from decode_gemv_elementwise_amd import paged
from test_gpu_paged import DTYPES, I32, Case, ints
from test_gpu_paged_many import COUNTERS, check_twice

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[(60, 3000), (1, 5000)], [(1, 1), (70, 70)], [(130, 2500)], [(3, 4000), (60, 90)]])
@pytest.mark.parametrize("window", [0, 700])
def test_tables_far_wider_than_the_keys(lens, window):
    """2^31 keys fit the table: the plan counts more than one block as one, and the last keys have no place."""
    c = Case(lens, "bf16", 16, 8, 64, page=128, seed=7).poison_unused()
    c.window, c.sinks = window, 4
    y, bound, mine = paged_ref.attn(c.q, c.k, c.v, ints(c.table, "cpu"), ints(c.starts, "cpu"), ints(c.lens, "cpu"), c.scale,
                                    window, 4, torch.bfloat16)
    assert mine.all()
    table = torch.full((len(lens), 1 << 24), -1, dtype=I32, device="cuda")
    table[:, :len(c.table[0])] = ints(c.table)
    first = None
    for _ in range(2):
        out = torch.full_like(c.q, 7.0)
        paged.gemv_paged_attn(c.q, c.k, c.v, table, ints(c.starts), ints(c.lens), c.scale, out, c.work, window=window, sinks=4)
        assert ((out.double().cpu() - y).abs() <= bound).all()
        assert first is None or out.equal(first), "another result the second time"
        first = out
        assert not c.work[:COUNTERS].any()


@pytest.mark.parametrize("dim", [64, 128])
def test_cut_tiles_past_the_first_requests(dim):
    """300 requests, short but for the last: few rows and many over thousands of keys, cut and joined."""
    lens = [(1, 3 + r % 5) for r in range(295)] + [(1, 6000), (0, 9), (40, 3000), (5, 2500), (1, 4001)]
    check_twice(Case(lens, "f16", 4, 2, dim, seed=8), "the last of 300 requests")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tokens_far_apart(dtype):
    """Pages of 16 whose tokens are 2^27 elements apart: offsets within a page past 32 bits of bytes."""
    c = Case([(20, 100), (1, 60)], dtype, 4, 2, 64, seed=9)
    shape = c.k.shape
    far = (2 * 64, 1 << 27, 64, 1)
    size = sum((n - 1) * s for n, s in zip(shape, far)) + 1
    k, v = (torch.empty(size, device="cuda", dtype=DTYPES[dtype]).as_strided(shape, far) for _ in "kv")
    k.copy_(c.k), v.copy_(c.v)
    c.k, c.v = k, v
    out = c.run()
    c.k, c.v = k.contiguous(), v.contiguous()
    c.check(out, "far")
