"""The example's attention block over a cache in 8 bits: prompts in chunks among single
tokens, through a captured graph and without."""
import os
import sys

import pytest
import torch

import paged8_ref as ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

STEPS = ([8, 0, 0], [1, 7, 0], [1, 1, 6], [1, 1, 1], [0, 8, 0], [1, 0, 4], [2, 2, 2], [1, 1, 1])


@pytest.mark.parametrize("codes", ref.CODES)
@pytest.mark.parametrize("window", [0, 6])
def test_steps(codes, window):
    """Every step's attention by its definition over what the cache holds, the same through a graph and without; what the
    cache holds is within its steps of what a cache of bfloat16 holds."""
    from paged_decode import Block

    make = lambda **more: Block(hidden=256, heads=4, kv_heads=2, dim=64, page=4, pages=64, requests=3, longest=64, window=window,  # noqa: E731
                                sinks=2, **more)
    eager, graph, wide = make(codes=codes), make(codes=codes), make()
    g = torch.Generator(device="cuda").manual_seed(1)
    for fresh in STEPS:
        n = sum(fresh)
        x = torch.randn(n, 256, generator=g, device="cuda")
        y = eager.step(x, list(fresh), False)
        assert graph.step(x, list(fresh), True).equal(y)
        wide.step(x, list(fresh), False)
        k, v, ks, vs = eager.cache
        want, bound, mine = ref.attn(eager.q[:n], k, ks, v, vs, eager.table, eager.query_start, eager.kv_len, 64 ** -0.5, window, 2,
                                     torch.float32)
        assert mine.all() and ((eager.mixed[:n].double().cpu() - want).abs() <= bound).all()
    assert all(a.view(torch.uint8).equal(b.view(torch.uint8)) for a, b in zip(eager.cache, graph.cache))
    for i, (codes_, scale) in enumerate(((k, ks), (v, vs))):
        got, full = ref.values(codes_, scale), wide.cache[i].double().cpu()
        step = ref.scales(scale.cpu())[..., None]  # of a page and head
        # rounded as a token came, and again whenever the scale grew: below a step in all (int8), half a step of its size
        # and the smallest (e4m3); bfloat16 is off by half a step 2^-8 itself
        tol = step if codes == "int8" else 2.0 ** -4 * full.abs() + 2.0 ** -9 * step
        for table, length in zip(eager.table.tolist(), eager.lengths):
            for j in range(length):
                at = table[j // 4], j % 4
                assert ((got[at] - full[at]).abs() <= (tol[at] if codes == "e4m3" else step[at[0], 0]) + 2.0 ** -8 * full[at].abs()).all()


@pytest.mark.parametrize("codes", ref.CODES)
def test_example_runs(codes, capsys):
    import paged_decode

    paged_decode.main(codes)
    assert "lengths [12, 10, 8, 6]" in capsys.readouterr().out
