"""The example's bookkeeping on the host: a step that is refused takes nothing."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def block(lengths, pool, longest):
    """A block's books without its buffers: a step that gets past them fails on those."""
    from paged_decode import Block

    b = Block.__new__(Block)
    b.hidden, b.page, b.longest, b.lengths, b.pool = 8, 4, longest, list(lengths), list(pool)
    return b


@pytest.mark.parametrize("lengths,pool,longest,fresh,what", [
    ([4, 8], [7], 64, [1, 1], "pages"), ([0, 0], [], 64, [0, 1], "pages"), ([3, 60], [5, 6, 7], 60, [0, 1], "longer"),
    ([3, 62], [5, 6, 7], 63, [1, 2], "longer")])
def test_a_refused_step_takes_nothing(lengths, pool, longest, fresh, what):
    b = block(lengths, pool, longest)
    with pytest.raises(ValueError, match=what):
        b.step(torch.zeros(sum(fresh), 8), fresh)
    assert b.pool == pool and b.lengths == lengths


def test_a_step_within_bounds_is_not_refused():
    b = block([3, 59], [5, 6], 60)
    with pytest.raises(AttributeError):  # the first buffer
        b.step(torch.zeros(2, 8), [1, 1])
