"""The operators over a paged cache in 8 bits at the far ends of the scales."""
import random

import pytest
import torch

import paged8_ref as ref
from test_gpu_paged8 import STEPS, Cache, Case, places, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("rot,shift", [(0, 0), (64, 0), (50, 0), (0, 1)])
def test_append_into_blocks_of_the_largest_scales(code, rot, shift):
    """Blocks whose scale is 2^123 to 2^127, the largest that a byte stands for, get values that are codes other than 0
    there: by the wide path one token and several at a time, and by the general one."""
    for byte in ((250, 255), (254, 255)):
        c = Cache(code, 8, 16, 16, 1, 64, seed=5, byte=byte)
        run_append(c, "f32", "bf16", [1, 2, 20, 37, 38, 39, 63], 1, rot, shift=shift, grow=2.0 ** 123)
        c = Cache(code, 20, 16, 16, 2, 64, seed=6, byte=byte)
        run_append(c, "f32", "bf16", places(random.Random(2), STEPS["tokens"] + STEPS["drafts"], 16, 20), 2, rot, shift=shift,
                   grow=2.0 ** 122, seed=3)


@pytest.mark.parametrize("code", ref.CODES)
@pytest.mark.parametrize("lens", [[(1, 2000)], [(40, 2000)]])
@pytest.mark.parametrize("byte", [12, 20, 30, 60, 200])
def test_small_weights_beside_far_scales(code, lens, byte):
    """One key takes nearly all of the weight and has a v of 0, so the result is what 2000 weights of about 2^-22 give,
    under scales of v near the least and far from it.  A part w v below 2^-117 (448 steps of the least normal number) may
    be taken as 0, and no other: 2000 such parts at most, beside the bound of any call."""
    c = Case(lens, code, "bf16", 2, 1, 64, seed=byte)
    v = c.c.v.float().abs().clamp(min=1.0)  # all of one sign: no sum is smaller than its parts
    c.c.v.copy_(v.to(c.c.v.dtype))
    c.c.vs.fill_(byte)
    c.c.k.zero_()
    c.c.ks.fill_(127)
    c.c.k[c.table[0][0], 5, 0, 0] = 64
    c.c.v[c.table[0][0], 5] = 0
    c.q.zero_()
    c.q[..., 0] = 1.921875  # scores of 1.921875 64 / 8 = 15.375 and 0: weights of e^-15.375 = 2^-22.2
    for out_type in (torch.bfloat16, torch.float32):
        y, bound, mine = c.want(out_type)
        got = c.run(out_type).double().cpu()
        assert mine.all() and (y[:, :, 0] > 0).all()
        err = (got - y).abs() - bound
        assert float(err.max()) <= 2000 * 2.0 ** -117, f"off by {float(err.max()):.3e} beyond the bound"
        if byte > 30:  # every part is far above: nothing is lost
            assert float(err.max()) <= 0
