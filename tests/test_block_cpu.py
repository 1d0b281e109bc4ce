"""The C entry points of group norm, gated recurrence and gated linear units without a GPU: sizes of workspaces and
refusals before any launch."""
import ctypes
import math

import pytest

from helpers import ensure_built

torch = pytest.importorskip("torch")

ARG, EMPTY, SHAPE, WORKSPACE, TOO_LARGE = 1, 3, 4, 5, 8
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    from differentiable_series_alignment_gb300 import _lib
    _lib.load()
    return _lib


def norm_calls(lib, x=0x1000, y=0x2000, mean=0x3000, rstd=0x4000, B=2, S=3, G=2, C=8, eps=1e-5, activation=1, dtype=0, wdtype=0, ws=0x100000,
               ws_bytes=1 << 50, dx=0x5000, dw=0x6000):
    f = lib.load()
    yield f.sdtw_groupnorm_forward(vp(x), None, None, None, B, S, G, C, eps, activation, dtype, wdtype, vp(y), vp(mean), vp(rstd), vp(ws),
                                   ws_bytes, None)
    yield f.sdtw_groupnorm_backward(vp(y), vp(x), None, None, None, vp(mean), vp(rstd), B, S, G, C, activation, dtype, wdtype, vp(dx), vp(dw),
                                    None, vp(ws), ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=0), EMPTY), (dict(S=0), EMPTY), (dict(G=0), EMPTY), (dict(C=0), EMPTY), (dict(C=7), SHAPE), (dict(dtype=3), ARG),
    (dict(wdtype=-1), ARG), (dict(activation=4), ARG), (dict(activation=-1), ARG), (dict(x=None), ARG), (dict(y=None), ARG),
    (dict(mean=None), ARG), (dict(rstd=None), ARG), (dict(B=1 << 30, G=8), TOO_LARGE),
    (dict(B=(1 << 30) + 1, G=1), TOO_LARGE), (dict(C=1 << 25), TOO_LARGE)])
def test_group_norm_refusals(lib, change, code):
    assert list(norm_calls(lib, **change)) == [code, code]
    if code in (EMPTY, SHAPE, TOO_LARGE) or "dtype" in change:
        size = dict(B=2, S=3, G=2, C=8, dtype=0)
        size.update({k: v for k, v in change.items() if k in size})
        f = lib.load()
        assert f.sdtw_groupnorm_workspace_bytes(*size.values(), 0) == 0 and f.sdtw_groupnorm_workspace_bytes(*size.values(), 1) == 0


def test_group_norm_refuses_eps_and_workspaces(lib):
    for eps in (-1.0, math.nan, math.inf):
        assert next(norm_calls(lib, eps=eps)) == ARG
    assert lib.load().sdtw_groupnorm_workspace_bytes(2, 3, 2, 8, 0, 1) > 0
    for bad in (dict(ws=None), dict(ws=0x100008), dict(ws_bytes=8)):
        assert list(norm_calls(lib, **bad))[1] == WORKSPACE
    assert lib.load().sdtw_groupnorm_backward(vp(1), vp(1), None, None, None, vp(1), vp(1), 2, 3, 2, 8, 0, 0, 0, None, None, None, None, 0,
                                              None) == 0     # nothing is asked for


@pytest.mark.parametrize("change,code", [
    (dict(B=0), EMPTY), (dict(N=0), EMPTY), (dict(C=0), EMPTY), (dict(x=None), ARG), (dict(gate=None), ARG), (dict(dtype=5), ARG),
    (dict(N=1 << 30, C=1), TOO_LARGE), (dict(C=(1 << 30) + 1), TOO_LARGE),
    (dict(x_stride=(64, (1 << 23) + 1)), TOO_LARGE), (dict(gate_stride=(64, -(1 << 24))), TOO_LARGE),
    (dict(x_stride=(64, -(1 << 63))), TOO_LARGE)])
def test_recurrence_refusals(lib, change, code):
    base = dict(x=0x1000, gate=0x2000, x_stride=(64, 8), gate_stride=(64, 8), state=None, lengths=None, B=2, N=3, C=8, dtype=0, reverse=0, tied=1)
    base.update(change)
    p = lib.Recurrence(*base.values())
    f = lib.load()
    assert f.sdtw_recurrence_forward(ctypes.byref(p), vp(0x3000), None, None, None) == code
    assert f.sdtw_recurrence_backward(ctypes.byref(p), vp(0x3000), None, None, vp(0x4000), vp(0x5000), None, None) == code


def test_recurrence_refuses_missing_results(lib):
    p = lib.Recurrence(0x1000, 0x2000, (64, 8), (64, 8), None, None, 2, 3, 8, 0, 0, 1)
    f = lib.load()
    assert f.sdtw_recurrence_forward(None, vp(1), None, None, None) == ARG
    assert f.sdtw_recurrence_forward(ctypes.byref(p), None, None, None, None) == ARG
    for kept, dx, dgate in ((None, 1, 1), (1, None, 1), (1, 1, None)):
        assert f.sdtw_recurrence_backward(ctypes.byref(p), vp(kept), None, None, vp(dx), vp(dgate), None, None) == ARG


def gated(lib, **change):
    base = dict(x=0x1000, gate_weight=0x2000, up_weight=0x3000, gate_bias=None, up_bias=None, x_stride=64, gate_stride=64, up_stride=64, R=200,
                K=64, F=128, dtype=1, activation=1)
    base.update(change)
    return lib.Gated(*base.values())


@pytest.mark.parametrize("change,code", [
    (dict(R=0), EMPTY), (dict(K=0), EMPTY), (dict(F=0), EMPTY), (dict(x=None), ARG), (dict(up_weight=None), ARG), (dict(gate_weight=None), ARG),
    (dict(R=1 << 30, F=1 << 10), TOO_LARGE), (dict(dtype=9), ARG), (dict(activation=0), ARG), (dict(activation=5), ARG), (dict(R=1 << 40), TOO_LARGE), (dict(K=1 << 24), TOO_LARGE),
    (dict(F=1 << 24), TOO_LARGE)])
def test_gated_refusals(lib, change, code):
    p = gated(lib, **change)
    f = lib.load()
    assert f.sdtw_gated_forward(ctypes.byref(p), vp(0x4000), vp(0x100000), 1 << 50, None) == code
    assert f.sdtw_gated_backward(ctypes.byref(p), vp(0x4000), vp(0x5000), None, None, None, None, vp(0x100000), 1 << 50, None) == code
    assert lib.sdtw_gated_workspace_bytes(p) == 0 and lib.sdtw_gated_workspace_bytes(p, True) == 0


def test_gated_refuses_missing_results_and_workspaces(lib):
    f, p = lib.load(), gated(lib)
    assert f.sdtw_gated_forward(None, vp(0x4000), None, 0, None) == ARG
    assert f.sdtw_gated_forward(ctypes.byref(p), None, vp(0x100000), 1 << 50, None) == ARG
    back = lambda dh=0x4000, dx=0x5000, ws=0x100000, n=1 << 50: f.sdtw_gated_backward(  # noqa: E731
        ctypes.byref(p), vp(dh), vp(dx), None, None, None, None, vp(ws), n, None)
    assert back(dh=None) == ARG and back(dx=None) == 0
    assert lib.sdtw_gated_workspace_bytes(p, True) > 0
    assert back(ws=None) == WORKSPACE and back(ws=0x100010) == WORKSPACE and back(n=64) == WORKSPACE


def test_slabs_of_a_prime_number_of_channels_are_chosen_quickly(lib):
    """The width of a slab is looked for among those that a CTA can have, not up to the channels, by which 100 calls took 12 s."""
    import time
    start = time.monotonic()
    for _ in range(100):
        assert lib.load().sdtw_groupnorm_workspace_bytes(1, 2, 16777213, 16777213, 1, 1) == 2 * 16777213 * 4
    assert time.monotonic() - start < 2.0
