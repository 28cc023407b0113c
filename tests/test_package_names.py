"""What the package names is there, and every module of operators is named."""
import importlib

import pytest

pytest.importorskip("torch")

import decode_gemv_elementwise_amd as package


def test_every_module_of_operators_is_named():
    assert {"binding", "paged", "paged8"} <= set(package.__all__)
    for name in package.__all__:
        importlib.import_module(f"{package.__name__}.{name}")
