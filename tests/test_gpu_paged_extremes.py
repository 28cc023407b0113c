"""The paged attention at scores far beyond a trained head's, and at infinities
and NaN of v beside a result in 32 bits, in rows few and many."""
import math

import pytest
import torch

from paged_ref import HALF_STEP
from test_gpu_paged import DTYPES, Case

pytestmark = pytest.mark.gpu

# a tile of few rows, one of many, and both cut over workgroups
LENS = {"few": [(1, 1), (1, 40), (3, 70)], "many": [(20, 20), (20, 70)], "few_cut": [(1, 3000)], "many_cut": [(20, 2000)]}


def rows_of(c):
    """(row of q, request, its position) of every new token."""
    for r, kv in enumerate(c.lens):
        q0, n = c.starts[r], c.starts[r + 1] - c.starts[r]
        for i in range(n):
            yield q0 + i, r, kv - n + i


def key(c, t, r, j):
    return t[c.table[r][j // c.page], j % c.page]


def keys_of(c, t, r):
    """[keys, heads, dim] of request r."""
    j = torch.arange(c.lens[r])
    return t[torch.tensor(c.table[r])[j // c.page], j % c.page]


def held(c, want, out_dtype, slack=0.0):
    """The result against `want` [tokens, heads, dim] where the weights are exact: the f32 sums over n keys (n 2^-24
    of the mean |v|, below 6) and the result's own half step, and `slack` of the mean |v| beside them."""
    out = c.run(out_dtype).double().cpu()
    assert torch.isfinite(out).all(), f"{int((~torch.isfinite(out)).sum())} of {out.numel()} values are not finite"
    bound = HALF_STEP[out_dtype] * want.abs() * 1.01 + 6 * ((max(c.lens) + 8) * 2.0 ** -24 + slack)
    worst = float(((out - want).abs() - bound).max())
    assert worst <= 0, f"beyond the bound by {worst:.3e}"


@pytest.mark.parametrize("dtype,size", [("f16", s) for s in (700, 1800, 1900, 2200, 3000, 4000, 20000)] +
                         [("bf16", s) for s in (4000.0, 1e6, 1e9, 1e15)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_equal_keys_of_any_size(dtype, size, dim):
    """Keys that are all alike weigh alike, however large their scores: the mean of v."""
    for lens in LENS:
        c = Case(LENS[lens], dtype, 2, 1, dim, seed=3)
        c.q[:], c.k[:] = size, size
        want = torch.zeros(c.q.shape, dtype=torch.float64)
        v = [keys_of(c, c.v.cpu().double(), r) for r in range(len(c.lens))]
        for row, r, p in rows_of(c):
            want[row] = v[r][:p + 1].mean(0)
        for out in (c.q.dtype, torch.float32):
            held(c, want, out)


@pytest.mark.parametrize("dtype,size", [("f16", 16.0), ("f16", 2000.0), ("bf16", 16.0), ("bf16", 1e12)])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("dim", [64, 256])
def test_one_key_far_above_the_others(dtype, size, rising, dim):
    """Scores that rise (or fall) by more than 2^10 a key: the largest that a row sees is all of its result."""
    for lens in LENS:
        c = Case(LENS[lens], dtype, 2, 1, dim, seed=4)
        top, k = max(c.lens), torch.zeros_like(c.k, device="cpu")
        c.q[:] = 0
        c.q[..., 0], c.q[..., 1] = size, size
        # two values make the rank, which one of 8 bits would not
        for r, kv in enumerate(c.lens):
            for j in range(kv):
                rank = j + 1 if rising else top - j
                key(c, k, r, j)[..., 0] = rank // 64 * 64
                key(c, k, r, j)[..., 1] = rank % 64
        c.k = k.cuda()
        c.scale = 2.0 ** 10 / size
        want = torch.zeros(c.q.shape, dtype=torch.float64)
        v = c.v.cpu().double()
        for row, r, p in rows_of(c):
            want[row] = key(c, v, r, p if rising else 0)
        for out in (c.q.dtype, torch.float32):
            held(c, want, out)


def test_steps_of_the_score_above_the_slack():
    """Scores of 2^24, where a step of 32 bits is 2: the running maximum's slack of 1 must not let a weight of 2^2
    pass, which binary16 does not hold when lifted."""
    scale = float(torch.tensor(math.log(2.0), dtype=torch.float32))  # times log2(e) it is 1 in 32 bits
    for lens in ([(20, 400)], [(2, 400)]):
        c = Case(lens, "f16", 2, 1, 64, seed=5)
        c.q[:], c.k[:] = 0, 0
        c.q[..., 0], c.q[..., 1] = 4096, 1
        c.k[..., 0] = 4096
        c.scale = scale
        v = keys_of(c, c.v.cpu().double(), 0)
        step = [2 + 2 * (j // 64) for j in range(400)]
        for j in range(400):
            key(c, c.k, 0, j)[..., 1] = step[j]
        want = torch.zeros(c.q.shape, dtype=torch.float64)
        for row, _, p in rows_of(c):
            w = torch.tensor([2.0 ** (step[j] - step[p]) for j in range(p + 1)], dtype=torch.float64)
            want[row] = (w[:, None, None] * v[:p + 1]).sum(0) / w.sum()
        held(c, want, torch.float16)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_special_values_in_float32_results(value, dtype, dim):
    """An infinity or NaN of v in keys that all rows see, that some see, and behind the window."""
    for window in (0, 300):
        c = Case([(40, 1200), (3, 500), (1, 2000), (1, 1)], dtype, 2, 1, dim, seed=5)
        c.window, c.sinks = window, 3
        for r, j in ((0, 20), (0, 1175), (1, 470), (1, 1), (2, 40), (2, 1990), (3, 0)):
            key(c, c.v, r, j)[0, 7 + j % 3] = value
        c.check(c.run(torch.float32), f"{value} window {window}")


def test_infinities_beside_weights_that_binary16_does_not_hold():
    """An infinity whose weight is 2^-57 of the largest: itself or NaN in every row that sees its key, by where in the
    row that lies, and nothing of it in the other rows."""
    for lens, at in (([(1, 40), (1, 40)], (3, 39)), ([(20, 100), (20, 100)], (3, 85))):
        c = Case(lens, "f16", 2, 1, 64, seed=6)
        c.q[:], c.k[:] = 0, 0
        c.q[..., 0] = 8
        for r in range(2):
            key(c, c.k, r, 10)[..., 0] = 40  # a score of 40, the others' is 0
            key(c, c.v, r, at[r])[..., 9] = float("inf")
        want = torch.zeros(c.q.shape, dtype=torch.bool)
        for row, r, p in rows_of(c):
            want[row, :, 9] = p >= at[r]
        for out in (torch.float16, torch.float32):
            got = c.run(out).cpu()
            assert torch.isfinite(got).equal(~want), f"{lens} {out}"
            assert not (got == float("-inf")).any()
