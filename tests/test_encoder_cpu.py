"""The encoder operators' C entry points without a GPU: sizes of workspaces and refusals before any launch, and
the rotary tables against their formulas."""
import ctypes
import math

import pytest

from helpers import ensure_built

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    from differentiable_series_alignment_gb300 import _lib
    _lib.load()
    return _lib


ARG, EMPTY, SHAPE, WORKSPACE, TOO_LARGE = 1, 3, 4, 5, 8


def problem(lib, **change):
    base = dict(q=0x1000, k=0x2000, v=0x3000, q_stride=(64, 64, 64), k_stride=(64, 64, 64), v_stride=(64, 64, 64),
                q_lengths=None, k_lengths=None, B=2, N=3, M=5, Hq=4, Hkv=2, D=16, dtype=0, window_left=-1, window_right=-1,
                scale=1.0)
    base.update(change)
    return lib.Attention(*base.values())


@pytest.mark.parametrize("change,code", [
    (dict(B=0), EMPTY), (dict(N=0), EMPTY), (dict(M=0), EMPTY), (dict(Hkv=0), EMPTY), (dict(D=0), EMPTY), (dict(Hq=3), SHAPE),
    (dict(q=None), ARG), (dict(v=None), ARG), (dict(dtype=3), ARG), (dict(window_left=-2), ARG), (dict(scale=0.0), ARG),
    (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(D=129), TOO_LARGE), (dict(M=1 << 29), TOO_LARGE),
    (dict(N=1 << 28), TOO_LARGE), (dict(B=1 << 27, N=1024), TOO_LARGE)])
def test_attention_refusals(lib, change, code):
    p = problem(lib, **change)
    f = lib.load()
    vp = ctypes.c_void_p
    assert f.sdtw_attention_forward(ctypes.byref(p), vp(0x4000), None, None, vp(0x100000), 1 << 40, None) == code
    assert f.sdtw_attention_backward(ctypes.byref(p), vp(0x4000), None, vp(0x5000), vp(0x6000), vp(0x7000), vp(0x8000),
                                     vp(0x9000), vp(0x100000), 1 << 40, None) == code
    assert lib.sdtw_attention_workspace_bytes(p) == 0 and lib.sdtw_attention_workspace_bytes(p, True) == 0


def test_attention_refuses_missing_results_and_workspaces(lib):
    f, vp = lib.load(), ctypes.c_void_p
    p = problem(lib)
    assert f.sdtw_attention_forward(None, vp(0x4000), None, None, None, 0, None) == ARG
    assert f.sdtw_attention_forward(ctypes.byref(p), None, None, None, vp(0x100000), 1 << 40, None) == ARG
    back = lambda out=0x4000, lse=0x5000, do=0x6000, dq=0x7000, dk=0x8000, dv=0x9000, ws=0x100000, n=1 << 40: (  # noqa: E731
        f.sdtw_attention_backward(ctypes.byref(p), vp(out), None, vp(lse), vp(do), vp(dq), vp(dk), vp(dv), vp(ws), n, None))
    assert back(out=None) == ARG and back(lse=None) == ARG and back(do=None) == ARG
    assert back(dk=None) == ARG and back(dv=None) == ARG          # both or neither
    assert back(ws=None) == WORKSPACE and back(ws=0x100008) == WORKSPACE and back(n=64) == WORKSPACE
    assert back(dq=None, dk=None, dv=None) == 0                    # nothing is asked for
    few = problem(lib, N=1, M=100000)                              # a split key axis needs room for its parts
    assert lib.sdtw_attention_workspace_bytes(few) > 0
    assert f.sdtw_attention_forward(ctypes.byref(few), vp(0x4000), None, None, None, 0, None) == WORKSPACE


def test_workspace_sizes(lib):
    rows = 2 * 2 * 128 * 4                                         # B Hkv (N G rounded up to 128) floats
    assert lib.sdtw_attention_workspace_bytes(problem(lib), True) >= 2 * rows
    assert lib.sdtw_attention_workspace_bytes(problem(lib, B=64, N=4096)) == 0
    assert lib.sdtw_layernorm_workspace_bytes(1000, 64) >= 2 * 4 * 64
    assert lib.sdtw_layernorm_workspace_bytes(0, 64) == 0 and lib.sdtw_layernorm_workspace_bytes(5, 0) == 0


def test_norm_refusals(lib):
    f, vp = lib.load(), ctypes.c_void_p
    go = lambda x=0x1000, rows=4, C=8, eps=1e-5, dt=0, wdt=0, y=0x2000, mean=0x3000, rstd=0x4000: (  # noqa: E731
        f.sdtw_layernorm_forward(vp(x), None, None, rows, C, eps, dt, wdt, vp(y), vp(mean), vp(rstd), None))
    assert go(rows=0) == EMPTY and go(C=0) == EMPTY
    assert go(x=None) == ARG and go(y=None) == ARG and go(dt=5) == ARG and go(wdt=-1) == ARG
    assert go(mean=None) == ARG and go(eps=-1.0) == ARG and go(eps=math.nan) == ARG
    assert go(C=(1 << 24) + 1) == TOO_LARGE
    back = lambda dy=0x1000, mean=0x3000, dw=0x5000, ws=0x100000, n=1 << 30: (  # noqa: E731
        f.sdtw_layernorm_backward(vp(dy), vp(0x2000), None, vp(mean), vp(0x4000), 4, 8, 0, 0, None, vp(dw), None, vp(ws), n, None))
    assert back(dy=None) == ARG and back(mean=None) == ARG
    assert back(ws=None) == WORKSPACE and back(n=8) == WORKSPACE and back(ws=0x100004) == WORKSPACE
    assert back(dw=None, ws=None) == 0


def test_rotary_refusals(lib):
    f, vp = lib.load(), ctypes.c_void_p
    st = (ctypes.c_longlong * 3)(64, 64, 64)
    go = lambda q=0x1000, k=0x2000, ko=0x3000, B=1, N=4, D=16, R=8, table=0x4000, length=8, pos=None, ps=0, dt=0, qs=st: (  # noqa: E731
        f.sdtw_rotary(vp(q), qs, vp(k), st, B, N, 2, 2, D, R, vp(table), length, vp(pos), ps, 0, 0, dt, vp(0x5000), vp(ko), None))
    assert go(B=0) == EMPTY and go(length=0) == EMPTY
    assert go(q=None) == ARG and go(table=None) == ARG and go(ko=None) == ARG and go(k=None) == ARG and go(dt=9) == ARG
    assert go(qs=None) == ARG
    assert go(R=7) == SHAPE and go(R=18) == SHAPE and go(R=0) == SHAPE
    assert go(N=9) == SHAPE and go(pos=0x6000, ps=2) == SHAPE


def test_rotary_tables():
    from differentiable_series_alignment_gb300 import rotary_table
    t = rotary_table(50, 8, device="cpu")
    assert t.shape == (50, 4, 2) and t.dtype == torch.float32
    for pos in (0, 1, 49):
        for i in range(4):
            a = pos * 10000.0 ** (-2 * i / 8)
            assert float(t[pos, i, 0]) == pytest.approx(math.cos(a), abs=2.0 ** -24)
            assert float(t[pos, i, 1]) == pytest.approx(math.sin(a), abs=2.0 ** -24)
    plain, linear = rotary_table(64, 16, device="cpu"), rotary_table(64, 16, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(linear[::4][:16], plain[:16], atol=1e-6, rtol=0)       # position 4 p turns like position p
    ntk = rotary_table(64, 16, scaling="ntk", factor=4.0, device="cpu")
    assert torch.equal(ntk[:, 0], plain[:, 0])                                    # the fastest pair as it was
    assert torch.allclose(ntk[::4][:16, -1], plain[:16, -1], atol=1e-6, rtol=0)  # the slowest stretched by the factor
    yarn = rotary_table(64, 64, scaling="yarn", factor=4.0, original_length=2048, device="cpu")
    m = 0.1 * math.log(4.0) + 1.0
    plain, linear = rotary_table(64, 64, device="cpu"), rotary_table(64, 64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(yarn[:, 0], plain[:, 0] * m, atol=1e-6, rtol=0)
    assert torch.allclose(yarn[:, -1], linear[:, -1] * m, atol=1e-6, rtol=0)
