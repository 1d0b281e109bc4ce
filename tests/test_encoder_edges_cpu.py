"""The encoder operators at the edges of their arguments, without a GPU: refusals of the C entry points before any launch, and the
rotary tables where their scalings begin and end."""
import ctypes

import pytest

from helpers import ensure_built

torch = pytest.importorskip("torch")

OK, ARG = 0, 1


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    from differentiable_series_alignment_gb300 import _lib
    _lib.load()
    return _lib


@pytest.mark.parametrize("table", [0x4001, 0x4002, 0x4004, 0x400c])
def test_rotary_refuses_a_table_off_eight_bytes(lib, table):
    """A pair's cosine and sine are one load."""
    vp, stride = ctypes.c_void_p, (ctypes.c_longlong * 3)(64, 64, 64)
    assert lib.load().sdtw_rotary(vp(0x1000), stride, None, None, 1, 4, 2, 0, 16, 8, vp(table), 8, None, 0, 0, 0, 0, vp(0x5000), None,
                                  None) == ARG
