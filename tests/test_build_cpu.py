"""The build: the C library stands on nvcc alone, and programs find it where they were linked to it."""
import ctypes
import importlib
import os
import shutil
import subprocess
import sys

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


def test_a_program_linked_by_path_starts(tmp_path):
    """gcc main.c path/to/libsdtw.so, run from anywhere without a search path."""
    library = ensure_built()
    (tmp_path / "main.c").write_text('#include "sdtw.h"\n#include <stdio.h>\n'
                                     'int main(void) { printf("%s", sdtw_status_string(SDTW_ERR_SHAPE)); return 0; }\n')
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    subprocess.run([gcc, "-I" + os.path.join(ROOT, "include"), str(tmp_path / "main.c"), library, "-o", str(tmp_path / "main")], check=True)
    clean = {k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"}
    r = subprocess.run([str(tmp_path / "main")], capture_output=True, text=True, env=clean, cwd=tmp_path)
    assert r.returncode == 0 and r.stdout, r.stderr


def test_the_binding_uses_the_library_beside_it():
    pytest.importorskip("torch")
    library = ensure_built()
    code = ("from differentiable_series_alignment_gb300 import _lib; _lib.binding()\n"
            "print({l.split()[-1] for l in open('/proc/self/maps') if l.rstrip().endswith('/libsdtw.so')})")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == str({os.path.realpath(library)}), r.stdout + r.stderr
