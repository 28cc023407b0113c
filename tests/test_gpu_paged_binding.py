"""The paged operators' calls from Python on the GPU: without the module that
marshals their tensors."""
import sys

import pytest
import torch

import decode_gemv_elementwise_amd as package
from decode_gemv_elementwise_amd import paged
from test_gpu_paged import Case, run_append, run_slots

pytestmark = pytest.mark.gpu


def test_calls_without_the_module(monkeypatch):
    """Every operator by the checks in Python alone: the same results."""
    c = Case([(1, 300), (9, 70)], "bf16")
    want = c.run()
    slots = ([5, 0, 33], [2, 0, 40], list(range(9)), 16, [[7, 8, 9, 0], [1, 2, 3, 4], [4, 5, 6, 0]], 60)
    want_slots = run_slots(*slots)
    monkeypatch.setitem(sys.modules, package.__name__ + "._paged_fast", None)
    monkeypatch.delattr(package, "_paged_fast", raising=False)
    for name in ("_LIB", "_FAST", "_DEVICE"):
        monkeypatch.setattr(paged, name, None)
    paged.load()
    assert paged._FAST is None
    assert c.run().equal(want)
    assert run_slots(*slots) == want_slots
    run_append("f32", "bf16", 9, 8, 2, 128, 128, 1, "halves", 16)
    with pytest.raises(TypeError):
        paged.gemv_paged_attn(c.q.float(), c.k, c.v, c.tt, c.qs, c.kl, 0.125, torch.empty_like(c.q), c.work)
