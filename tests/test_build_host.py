"""The build: the library alone where there is no torch."""

import importlib.util

import pytest


@pytest.fixture()
def B():
    from paged_kv_attention_slot_gb300 import build

    return build


def test_without_torch_the_library_is_built_alone(B, monkeypatch):
    real = importlib.util.find_spec
    assert B._binding_job(B._nvcc(), True) is not None
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert B._binding_job(B._nvcc(), True) is None
    assert B.build() == B.LIB
