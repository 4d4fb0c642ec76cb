"""What the build does beside compiling (no GPU needed): the library and the
module of the calls on PyTorch tensors do not wait for each other."""

import importlib.util
import os

import pytest

from kimi_delta_attention_kda_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's results in a folder of their own (objects stay where they are)."""
    build.build()
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(build, "TORCH_PATH", str(tmp_path / "_kda_torch.so"))
    return tmp_path


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_builds_without_pytorch(elsewhere, monkeypatch, capsys):
    without_torch(monkeypatch)
    assert build.build() == str(elsewhere / "libkda.so")
    assert os.listdir(elsewhere) == ["libkda.so"]
    assert "PyTorch" in capsys.readouterr().err


def test_the_library_builds_with_a_pytorch_without_cuda(elsewhere, monkeypatch):
    torch = elsewhere / "torch"
    (torch / "lib").mkdir(parents=True)
    find = importlib.util.find_spec
    spec = importlib.util.spec_from_file_location("torch", None, submodule_search_locations=[str(torch)])
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    build.build()
    assert (elsewhere / "libkda.so").exists() and not (elsewhere / "_kda_torch.so").exists()


def test_a_module_that_does_not_compile_leaves_the_library(elsewhere, monkeypatch):
    monkeypatch.setattr(build, "_torch_command", lambda *a: ["false"])
    with pytest.raises(RuntimeError, match="kda_torch.cpp"):
        build.build()
    assert (elsewhere / "libkda.so").exists() and not (elsewhere / "_kda_torch.so").exists()


def test_operators_name_the_missing_module(elsewhere, monkeypatch):
    from kimi_delta_attention_kda_gb300 import _lib
    build.build()
    monkeypatch.setattr(_lib, "_torch_module", None)
    monkeypatch.setattr(_lib, "TORCH_PATH", str(elsewhere / "not_there.so"))
    with pytest.raises(RuntimeError, match="not built"):
        _lib.load_torch_module()
