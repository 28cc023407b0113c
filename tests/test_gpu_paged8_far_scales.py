"""The operators over a paged cache in 8 bits at the far ends of the scales."""
import random

import pytest

import paged8_ref as ref
from test_gpu_paged8 import STEPS, Cache, places, run_append

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
