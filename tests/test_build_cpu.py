"""When the C++ binding has to be built again."""
from __future__ import annotations

import importlib.metadata
import os
import sys

import pytest

from quantized_swiglu_mlp_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_a_built_binding_stays(monkeypatch):
    assert not build._native_stale()


def test_another_torch_or_python_needs_another_binding(monkeypatch):
    real = importlib.metadata.version
    with monkeypatch.context() as m:
        m.setattr(importlib.metadata, "version", lambda name: "0.1" if name == "torch" else real(name))
        assert build._native_stale()
    with monkeypatch.context() as m:
        m.setattr(sys.implementation, "cache_tag", "cpython-0")
        assert build._native_stale()
    assert not build._native_stale()


def test_newer_sources_need_another_binding(monkeypatch):
    real = os.path.getmtime
    monkeypatch.setattr(os.path, "getmtime", lambda p: real(p) + (1e6 if p == build.NATIVE_SOURCE else 0))
    assert build._native_stale()
