"""What build() compiles, and when: with the compilers and torch replaced by stand-ins."""
import importlib.util
import os
import types

import pytest
import torch

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


@pytest.mark.parametrize("version", ["0.1.2", torch.__version__ + ".more"])
def test_another_torch_gets_an_extension_of_its_own(fresh, monkeypatch, tmp_path, version):
    """Whatever its files' age: the extension holds the layout of the torch it was built for."""
    (tmp_path / "version.py").write_text(f"__version__ = '{version}'\n")
    os.utime(tmp_path / "version.py", (1, 1))
    found = importlib.util.find_spec
    other = types.SimpleNamespace(submodule_search_locations=[str(tmp_path)])
    monkeypatch.setattr(libbuild.importlib.util, "find_spec",
                        lambda name, *a: other if name == "torch" else found(name, *a))
    monkeypatch.setattr(libbuild, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    with pytest.raises(AssertionError, match="started g"):
        libbuild.build()


def test_the_binding_takes_the_extension_of_its_torch():
    libbuild.build()
    assert os.path.exists(libbuild.torch_lib(torch.__version__))
    assert libbuild.torch_lib("2.9.1+cu130") != libbuild.torch_lib("2.9.1+cu128")
