"""The paged operators' calls from Python on the GPU: without the module that
marshals their tensors, and beside other threads."""
import ctypes
import subprocess
import sys
import threading
import time

import pytest
import torch

import decode_gemv_elementwise_amd as package
from decode_gemv_elementwise_amd import paged
from test_gpu_paged import Case, ints, run_append, run_slots

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


# stands in for a launch that waits: 0 once another thread has set `go`, -99 if none does for three seconds
WAITS = r"""
#include <unistd.h>
volatile int entered, go;
int launch(void)
{
    entered = 1;
    for (int i = 0; i < 3000 && !go; ++i)
        usleep(1000);
    return go ? 0 : -99;
}
"""


def test_other_threads_run_during_a_launch(tmp_path, monkeypatch):
    """A launch that waits for room in its stream's queue does not hold the interpreter."""
    paged.load()
    if paged._FAST is None:
        pytest.skip("the module is not built")
    (tmp_path / "waits.c").write_text(WAITS)
    lib = str(tmp_path / "waits.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", lib, str(tmp_path / "waits.c")], check=True, timeout=60)
    waits = ctypes.CDLL(lib)
    entered, go = (ctypes.c_int.in_dll(waits, n) for n in ("entered", "go"))

    def other():
        end = time.monotonic() + 10
        while not entered.value and time.monotonic() < end:
            time.sleep(0.001)
        go.value = 1

    c = Case([(1, 30)], "f16", 2, 1, 64)
    out = torch.empty_like(c.q)
    table, starts, lens, x = ints(c.table), ints(c.starts), ints(c.lens), torch.randn(1, 1, 64, device="cuda")
    one = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, 1, 4, 2, 1, 1, 1, 1, 1)]
    launch = ctypes.cast(waits.launch, ctypes.c_void_p).value
    calls = (
        lambda: paged.gemv_paged_slots(one[0], one[1], one[2], 16, table, *one[3:]),
        lambda: paged.gemv_paged_append(x, x, x, one[0], x[0, 0, :32].contiguous(), one[1],
                                        torch.empty(1, 1, 64, device="cuda", dtype=torch.float16), c.k, c.v),
        lambda: paged.gemv_paged_attn(c.q, c.k, c.v, table, starts, lens, 0.125, out, c.work))
    paged._FAST.bind(launch, launch, launch)
    try:
        for call in calls:
            entered.value = go.value = 0
            thread = threading.Thread(target=other)
            thread.start()
            call()  # raises for -99
            thread.join()
            assert entered.value == 1
    finally:
        monkeypatch.setattr(paged, "_LIB", None)
        paged.load()  # the library's own launches again
    assert c.run().isfinite().all()
