"""Which packed rows of an attention problem see a tile of keys: the arithmetic of csrc/attn_range.h on the CPU, at small
sizes against a plain enumeration and at the largest sizes that the entry points take against unbounded integers."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from helpers import ROOT

CSRC = os.path.join(ROOT, "differentiable_series_alignment_gb300", "csrc")
SOURCE = """
#include "attn_range.h"
extern "C" void seeing(const sdtw_attention* a, int b, int j0, int j1, int G, int* out)
{
    const sdtw::RowRange r(*a, b);
    const auto rows = r.seeing(j0, j1, G);
    out[0] = rows.lo, out[1] = rows.hi, out[2] = r.row_lo(j0), out[3] = r.row_hi(j0), out[4] = r.first_row();
}
"""


@pytest.fixture(scope="module")
def seeing(tmp_path_factory):
    compiler = shutil.which("g++")
    if compiler is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("range")
    (at / "range.cpp").write_text(SOURCE)
    # signed overflow ends the program instead of passing as some number
    subprocess.run([compiler, "-shared", "-fPIC", "-O1", "-std=c++17", "-ftrapv", "-I" + CSRC, str(at / "range.cpp"), "-o", str(at / "range.so")],
                   check=True)
    lib = ctypes.CDLL(str(at / "range.so"))
    from differentiable_series_alignment_gb300._lib import Attention

    def call(N, M, G, left, right, n, m, j0, j1):
        ql, kl = (ctypes.c_int * 1)(n), (ctypes.c_int * 1)(m)
        a = Attention(q_lengths=ctypes.addressof(ql), k_lengths=ctypes.addressof(kl), B=1, N=N, M=M, Hq=G, Hkv=1, D=8, window_left=left,
                      window_right=right, scale=1.0)
        out = (ctypes.c_int * 5)()
        lib.seeing(ctypes.byref(a), 0, j0, j1, G, out)
        return tuple(out)
    return call


def expected(n, m, G, left, right, j0, j1):
    """In unbounded integers; n and m are within the limits already."""
    last = min(j1, m) - 1
    if j0 > last:
        return 0, 0
    lo = 0 if right < 0 else max(0, j0 - (m - n) - right)
    hi = n if left < 0 else min(n, last - (m - n) + left + 1)
    return (lo * G, hi * G) if lo < hi else (0, 0)


def test_against_an_enumeration(seeing):
    rng = random.Random(1)
    for _ in range(3000):
        N, M, G, tile = rng.randint(1, 9), rng.randint(1, 12), rng.randint(1, 3), rng.randint(1, 5)
        n, m = rng.randint(0, N), rng.randint(0, M)
        left, right = rng.choice([-1, 0, 1, 4, 30]), rng.choice([-1, 0, 1, 4, 30])
        j0 = rng.randrange(0, M)
        rows = [i for i in range(n)
                if any((left < 0 or j >= i + m - n - left) and (right < 0 or j <= i + m - n + right) for j in range(j0, min(j0 + tile, m)))]
        lo, hi, one_lo, one_hi, first = seeing(N, M, G, left, right, n, m, j0, j0 + tile)
        assert list(range(lo, hi)) == [i * G + g for i in rows for g in range(G)]
        assert 0 <= one_lo <= n and 0 <= one_hi <= n
        blind = [i for i in range(n) if not any((left < 0 or j >= i + m - n - left) and (right < 0 or j <= i + m - n + right) for j in range(m))]
        assert blind == list(range(first))


@pytest.mark.parametrize("M", [16778216, 1 << 25, 1 << 26, 1 << 27])
@pytest.mark.parametrize("N,G", [(1, 128), (1, 127), (3, 100), (1 << 20, 128), (1, 1 << 27), (1 << 27, 1)])
def test_the_largest_sizes_stay_within_the_rows(seeing, N, G, M):
    rng = random.Random(N + G + M)
    for tile in (64, 128):
        for _ in range(300):
            n, m = rng.choice([N, N // 2, 0, rng.randint(0, N)]), rng.choice([M, M // 2 + 1, 0, rng.randint(0, M)])
            left, right = rng.choice([-1, 0, 64, M, M + N - 1]), rng.choice([-1, 0, 64, M, M + N - 1])
            j0 = rng.choice([0, M // 2, M - 1, rng.randrange(M)]) // tile * tile
            lo, hi, one_lo, one_hi, first = seeing(N, M, G, left, right, n, m, j0, j0 + tile)
            assert (lo, hi) == expected(n, m, G, left, right, j0, j0 + tile)
            assert 0 <= one_lo <= n and 0 <= one_hi <= n and 0 <= first <= n


def test_old_keys_of_a_long_cache_are_seen_by_no_row(seeing):
    for M in (16778216, 1 << 25):
        for j0 in range(0, M - 10000, 64 * 997):
            assert seeing(1, M, 128, 64, 0, 1, M, j0, j0 + 64)[:2] == (0, 0)
        assert seeing(1, M, 128, 64, 0, 1, M, (M - 1) // 64 * 64, M)[:2] == (0, 128)
