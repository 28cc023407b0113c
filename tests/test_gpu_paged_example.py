"""The example's attention block against plain attention without a cache: prompts
in chunks among single tokens, through a captured graph and without."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

STEPS = ([8, 0, 0], [1, 7, 0], [1, 1, 6], [1, 1, 1], [0, 8, 0], [1, 0, 4], [2, 2, 2], [1, 1, 1])


def plain(block, xs):
    """Each request's whole sequence at once in 64 bits, q, k and v rounded as the block rounds them."""
    w_qkv, w_out = (torch.from_numpy(w.data).view(torch.bfloat16).view(n, -1).double()
                    for w, n in ((block.w_qkv, block.rows), (block.w_out, block.hidden)))
    d, out = block.dim, []
    for x in xs:
        x = x.double().cpu()
        q, k, v = (x @ w_qkv.t()).split([block.heads * d, block.kv_heads * d, block.kv_heads * d], 1)
        q, k, v = (t.unflatten(1, (-1, d)) for t in (q, k, v))
        angle = torch.arange(len(x)).double()[:, None] * block.inv_freq.double().cpu()
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        turn = lambda t: torch.cat([t[..., :d // 2] * c - t[..., d // 2:] * s, t[..., d // 2:] * c + t[..., :d // 2] * s], -1)  # noqa: E731
        q, k, v = (t.bfloat16().double() for t in (turn(q), turn(k), v))
        group = block.heads // block.kv_heads
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        p = torch.arange(len(x))
        seen = p[None, :] <= p[:, None]
        if block.window:
            seen &= (p[None, :] > p[:, None] - block.window) | (p[None, :] < block.sinks)
        score = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0).contiguous()) * d ** -0.5
        weight = torch.softmax(score.masked_fill(~seen, float("-inf")), -1)
        mixed = torch.matmul(weight, v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(len(x), -1)
        out.append(mixed @ w_out.t() + x)
    return out


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("window", [0, 6])
def test_steps_match_whole_sequences(graph, window):
    from paged_decode import Block

    block = Block(hidden=256, heads=4, kv_heads=2, dim=64, page=4, pages=64, requests=3, longest=64, window=window, sinks=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    xs, ys = [[], [], []], [[], [], []]
    for fresh in STEPS:
        x = torch.randn(sum(fresh), 256, generator=g, device="cuda")
        y = block.step(x, list(fresh), graph)
        at = 0
        for r, f in enumerate(fresh):
            xs[r].append(x[at:at + f])
            ys[r].append(y[at:at + f])
            at += f
    torch.cuda.synchronize()
    for r, want in enumerate(plain(block, [torch.cat(x) for x in xs])):
        got = torch.cat(ys[r]).double().cpu()
        # q, k and v round to bfloat16 after sums in 32 bits: at a border they may round the other way, a whole step
        # 2^-8 of a value; a score of size up to 8 then moves by 8 * 2 * 2^-8 in the rare worst case of all its terms,
        # and the mean of v (size about 1) over few keys by as much again
        assert float((got - want).abs().max()) < 16 * 2.0 ** -8, f"request {r}"
    held = [t for row, n in zip(block.table.tolist(), block.lengths) for t in row[:-(-n // 4)]]
    assert len(set(held)) == len(held) and sorted(held + block.pool) == list(range(64))
    free = len(block.pool)
    block.release(1)
    assert len(block.pool) == free + -(-20 // 4) and block.lengths[1] == 0


def test_example_runs(capsys):
    import paged_decode

    paged_decode.main()
    assert "lengths [12, 10, 8, 6]" in capsys.readouterr().out
