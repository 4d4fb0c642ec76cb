"""What the build does beside compiling (no GPU needed): the library and the
module of the calls on PyTorch tensors do not wait for each other, and the module
is only used with the PyTorch that it was built against."""

import importlib.util
import json
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


def test_another_pytorch_means_another_module(elsewhere, monkeypatch):
    monkeypatch.setattr(build, "TORCH_NOTE", str(elsewhere / "note.json"))
    compiled = []

    def command(torch_dir, target):
        # A stand-in for the compiler, which takes 20 seconds.
        compiled.append(target)
        return ["cp", os.path.join(build.CSRC, "kda_torch.cpp"), target] if ".tmp." in target else ["as", "before"]

    monkeypatch.setattr(build, "_torch_command", command)
    path = build.TORCH_PATH

    def builds():
        before = len([x for x in compiled if x != path])
        build.build()
        return len([x for x in compiled if x != path]) - before

    assert builds() == 1 and builds() == 0
    abi = build.torch_abi()
    assert "version" in abi["torch"] and json.load(open(build.TORCH_NOTE))["abi"] == abi
    for other in ({"torch": "__version__ = '0'"}, {"python": "cpython-99"}):
        monkeypatch.setattr(build, "torch_abi", lambda other=other: dict(abi, **other))
        assert builds() == 1 and builds() == 0
    os.remove(build.TORCH_NOTE)
    assert builds() == 1 and builds() == 0


@pytest.mark.parametrize("note", [None, {}, {"abi": {"torch": "__version__ = '0'", "python": "cpython-99"}}])
def test_a_module_for_another_pytorch_is_not_loaded(elsewhere, monkeypatch, note):
    from kimi_delta_attention_kda_gb300 import _lib
    monkeypatch.setattr(_lib, "_torch_module", None)
    monkeypatch.setattr(build, "TORCH_NOTE", str(elsewhere / "note.json"))
    if note is not None:
        (elsewhere / "note.json").write_text(json.dumps(note))
    with pytest.raises(RuntimeError, match="another PyTorch"):
        _lib.load_torch_module()
