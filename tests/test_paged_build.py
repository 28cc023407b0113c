"""The library is built, and the paged operators work, without the Python module
that marshals their tensors."""
import os
import subprocess
import sys

import pytest

from decode_gemv_elementwise_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def steps(monkeypatch):
    """build() with its compilations recorded in place of run."""
    done = []
    monkeypatch.setattr(build, "_compile", lambda sources, out, verbose: done.append(out) or out)
    monkeypatch.setattr(build, "build_cpu", lambda verbose=False: done.append(build.CPU_LIB))
    monkeypatch.setattr(build, "_run", lambda cmd, verbose: done.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: done.append(b))
    return done


def test_library_is_built_before_the_module(steps):
    pytest.importorskip("torch")
    assert build.build() == build.LIB
    assert steps.index(build.LIB) < steps.index(build.PY_LIB) == len(steps) - 1


def test_library_is_built_without_torch(steps, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert build.LIB in steps and build.CPU_LIB in steps and build.PY_LIB not in steps
    assert "torch" in capsys.readouterr().err


def test_library_is_built_without_a_cpp_compiler(steps, monkeypatch, capsys):
    pytest.importorskip("torch")
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build.build() == build.LIB
    assert build.LIB in steps and build.PY_LIB not in steps
    assert "g++" in capsys.readouterr().err


def test_module_is_named_for_its_interpreter():
    import importlib.machinery
    import sysconfig

    suffix = os.path.basename(build.PY_LIB)[len("_paged_fast"):]
    assert suffix == sysconfig.get_config_var("EXT_SUFFIX") and suffix in importlib.machinery.EXTENSION_SUFFIXES
    assert suffix not in (".so", ".abi3.so")


def test_paged_loads_without_the_module():
    """The checks and the refusals in Python serve where the module is missing."""
    pytest.importorskip("torch")
    if not os.path.exists(build.LIB):  # pragma: no cover - the build step makes it
        pytest.skip("the library is not built")
    code = """
import sys
sys.modules["decode_gemv_elementwise_amd._paged_fast"] = None
import torch
from decode_gemv_elementwise_amd import paged
assert paged.load() is not None and paged._FAST is None
assert paged.gemv_paged_attn_workspace(64) > 0
ints = lambda n: torch.zeros(n, dtype=torch.int32)
try:
    paged.gemv_paged_slots(ints(2), ints(2), ints(4), 16, ints(8).view(2, 4), ints(3), ints(2), ints(3), ints(3), ints(3), ints(1))
except TypeError as e:
    assert "GPU" in str(e)
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == "refused"


def test_cache_sizes_past_32_bits_are_refused():
    """The C structure's sizes are 32 bits wide: a larger one must not come out as another."""
    torch = pytest.importorskip("torch")
    from decode_gemv_elementwise_amd import paged

    if not os.path.exists(build.LIB):  # pragma: no cover - the build step makes it
        pytest.skip("the library is not built")
    paged.load()
    dev = torch.device("meta")
    for shape in ((1, 2 ** 32 + 16, 1, 8), (1, 16, 2 ** 32 + 1, 8), (1, 1, 1, 2 ** 32 + 64)):
        t = torch.empty(shape, dtype=torch.float16, device=dev)
        with pytest.raises(ValueError, match="2\\^31"):
            paged._cache_of(t, t, dev)
    t = torch.empty((2 ** 20, 16, 8, 128), dtype=torch.float16, device=dev)
    assert paged._cache_of(t, t, dev).num_pages == 2 ** 20
