"""What building the library needs, and what the Python layer does without the compiled binding."""
import importlib.util
import os

import pytest

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild


def test_the_library_is_built_without_torch(monkeypatch):
    libbuild.build()
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert libbuild.build() == libbuild.LIB_PATH
    assert libbuild.build_binding() is None


@pytest.mark.parametrize("missing", ["Python.h", "libtorch_python.so"])
def test_the_library_is_built_without_what_the_binding_needs(monkeypatch, missing):
    libbuild.build()
    there = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: there(p) and os.path.basename(p) != missing)
    assert libbuild.build() == libbuild.LIB_PATH
    assert libbuild.build_binding(force=True) is None
    assert there(libbuild.BINDING_PATH)          # one built before stays
