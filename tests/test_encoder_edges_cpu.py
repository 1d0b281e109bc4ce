"""The encoder operators at the edges of their arguments, without a GPU: refusals of the C entry points before any launch, and the
rotary tables where their scalings begin and end."""
import ctypes
import math

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


@pytest.mark.parametrize("dim,base,original", [(128, 1e4, 131072), (64, 1e4, 2048), (64, 1e4, 64), (64, 1e4, 4), (128, 5e5, 8192),
                                               (32, 1e4, 1 << 20)])
def test_yarn_divides_the_slow_pairs_alone(dim, base, original):
    """Pair by pair: how often it turns over the original length decides, wherever the ramp begins and ends."""
    from differentiable_series_alignment_gb300 import rotary_table
    factor, length = 4.0, 9
    plain = lambda i: base ** (-2.0 * i / dim)  # noqa: E731
    # real pair indices that turn beta_fast and beta_slow times
    fast, slow = (dim * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0))
    first, last = math.floor(fast), math.ceil(slow)
    magnitude = 0.1 * math.log(factor) + 1.0
    table = rotary_table(length, dim, base=base, scaling="yarn", factor=factor, original_length=original, device="cpu")
    for i in range(dim // 2):
        turns = original * plain(i) / (2 * math.pi)
        part = min(1.0, max(0.0, (i - first) / (last - first)))
        assert turns <= 32.0 or part == 0.0
        assert turns >= 1.0 or part == 1.0
        freq = plain(i) * (1 - part) + plain(i) / factor * part
        for p in range(length):
            # one rounding to fp32 of a value of at most `magnitude`
            assert float(table[p, i, 0]) == pytest.approx(magnitude * math.cos(p * freq), abs=2.0 ** -24 * magnitude + 1e-12)
            assert float(table[p, i, 1]) == pytest.approx(magnitude * math.sin(p * freq), abs=2.0 ** -24 * magnitude + 1e-12)


def test_rotary_table_goes_where_it_is_told(monkeypatch):
    """Device 0 by its number is a device, not the lack of one."""
    from differentiable_series_alignment_gb300 import encoder
    asked = []

    def arange(*args, device=None, **kwargs):
        asked.append(device)
        return real(*args, device="cpu", **kwargs)
    real = torch.arange
    monkeypatch.setattr(encoder.torch, "arange", arange)
    for device, want in ((0, 0), (None, "cuda"), ("cpu", "cpu")):
        asked.clear()
        encoder.rotary_table(4, 4, device=device)
        assert asked[0] == want


def test_rotary_table_refuses_ramps_that_go_nowhere():
    from differentiable_series_alignment_gb300 import rotary_table
    for fast, slow in ((1.0, 1.0), (1.0, 32.0), (32.0, 0.0), (32.0, -1.0), (math.nan, 1.0), (32.0, math.nan), (math.inf, 1.0)):
        with pytest.raises(ValueError, match="beta"):
            rotary_table(4, 8, scaling="yarn", factor=2.0, original_length=64, beta_fast=fast, beta_slow=slow, device="cpu")
    for bad in (dict(base=math.inf), dict(scaling="ntk", factor=math.inf), dict(scaling="linear", factor=math.nan)):
        with pytest.raises(ValueError):
            rotary_table(4, 8, device="cpu", **bad)
