"""What a build makes, in which order, and when it makes it again (CPU; the compilers
are stood in for)."""
import os
import sys

import pytest
import torch

from paged_kv_attention_partition_b200 import _build


@pytest.fixture
def package(tmp_path, monkeypatch):
    """An empty package folder, and compilers that write down what they are asked for."""
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libpad.so"))
    stale = _build.is_stale
    monkeypatch.setattr(_build, "is_stale", lambda: stale(str(tmp_path / "libpad.so")))
    if hasattr(_build, "BINDING"):
        monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_pad_torch.so"))
    made = []

    def compiler(name):
        def command(out, extra=()):
            made.append(name)
            return ["touch", out]
        return command

    monkeypatch.setattr(_build, "compile_command", compiler("library"))
    monkeypatch.setattr(_build, "binding_command", compiler("binding"))
    return made


def test_both_are_built_and_then_kept(package):
    assert os.path.exists(_build.build()) and package == ["library", "binding"]
    _build.build()
    assert package == ["library", "binding"]
    _build.build(force=True)
    assert package == ["library", "binding"] * 2


def test_the_library_does_not_wait_for_the_binding(package, monkeypatch):
    # the C library needs neither torch's headers nor g++
    monkeypatch.setattr(_build, "binding_command", lambda out: ["false"])
    with pytest.raises(RuntimeError):
        _build.build()
    assert os.path.exists(_build.LIB)


def test_without_torch_there_is_no_binding_to_build(package, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert os.path.exists(_build.build()) and package == ["library"]


def test_another_torch_gets_a_binding_of_its_own(package, monkeypatch):
    _build.build()
    monkeypatch.setattr(torch, "__version__", "99.0")
    _build.build()
    assert package == ["library", "binding", "binding"]
