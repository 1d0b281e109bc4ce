"""The build: the C library stands on nvcc alone, and programs find it where they were linked to it."""
import ctypes
import importlib
import os
import shutil
import subprocess

import pytest

from helpers import ROOT, ensure_built


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with one small source, all that it makes under tmp_path."""
    b = importlib.import_module("differentiable_series_alignment_gb300.build")
    source = tmp_path / "one.cu"
    source.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(b, "_sources", lambda: [str(source)])
    for name, value in (("BUILD", "objects"), ("LIB", "libsdtw.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / value))
    return b


def test_the_library_is_linked_where_the_binding_does_not_compile(build, monkeypatch):
    def fails(cc):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(build, "_binding_object", fails)
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):       # and the failure is told
        build.build(force=True)
    assert ctypes.CDLL(build.LIB).one() == 1 and not os.path.exists(build.BINDING)


def test_the_library_is_built_without_torch(build, monkeypatch, capsys):
    monkeypatch.setattr(build, "_has_torch", lambda: False)
    assert not build.up_to_date()
    assert build.build(force=True) == build.LIB
    assert ctypes.CDLL(build.LIB).one() == 1 and not os.path.exists(build.BINDING)
    assert "_binding.so" in capsys.readouterr().err
    assert build.up_to_date()
