"""What build() compiles, and when: with the compilers and torch replaced by stand-ins."""
import importlib.util
import os

import pytest

from block_sparse_attention_vsa_gb300 import build as libbuild


@pytest.fixture
def fresh(monkeypatch):
    """Everything is built; no nvcc from here on, and starting a compiler fails the test."""
    libbuild.build()

    def missing():
        raise RuntimeError("no nvcc")

    def started(cmd, **kw):
        raise AssertionError(f"started {cmd[0]}")

    monkeypatch.setattr(libbuild, "nvcc", missing)
    monkeypatch.setattr(libbuild.subprocess, "Popen", started)


def test_an_up_to_date_tree_needs_no_compiler(fresh):
    assert libbuild.build() == libbuild.LIB


def test_an_up_to_date_library_needs_no_torch(fresh, monkeypatch):
    found = importlib.util.find_spec
    monkeypatch.setattr(libbuild.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else found(name, *a))
    assert libbuild.build() == libbuild.LIB


def test_a_forced_build_asks_for_the_compiler(fresh):
    with pytest.raises(RuntimeError, match="no nvcc"):
        libbuild.build(force=True)
    assert os.path.exists(libbuild.LIB)
