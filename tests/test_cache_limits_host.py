"""Batches at the limits of what decode's counts hold, without a GPU: sizes that its ints do not count are refused."""
import ctypes
import subprocess

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

FAKE = 0x10000  # never dereferenced
INT_MAX = 2**31 - 1


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def workspace(L, rows, tiles, dtype=0, d=128):
    """Workspace bytes of one sequence with one head, `rows` new tokens and a table of `tiles` - 2 key tiles of 32."""
    c = fox.fox_cache(8, 32, 1, 1, d, dtype, FAKE, FAKE, FAKE, FAKE)
    b = fox.fox_batch(1, rows, tiles - 2, 0, FAKE, FAKE, FAKE, None)
    return L.fox_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), rows)


# dtype, d, rows of a row tile, workers, workers of a CTA
KERNELS = [(0, 128, 16, 608, 4), (0, 64, 16, 1216, 8), (1, 128, 8, 608, 4), (1, 64, 8, 1216, 4)]


@pytest.mark.parametrize("dtype,d,Rt,workers,warps", KERNELS)
def test_places_behind_the_line_s_end_are_ints_too(L, dtype, d, Rt, workers, warps):
    tiles = 1 << 16
    for row_tiles in (32767, 32760, 32600, 32500, 32400, 32000, 20000):
        total = tiles * row_tiles  # below 2^31 - workers, all of them
        assert total < INT_MAX - workers
        each = -(-total // workers)
        # the places that the kernels form before they cut them off: ends of a CTA's and of a worker's range
        most = max(total + warps * each, workers * each + each)
        size = workspace(L, row_tiles * Rt, tiles, dtype, d)
        if most > INT_MAX:
            assert size == 0, row_tiles
        if row_tiles <= 32000:
            assert most <= INT_MAX and size > 0
    c = fox.fox_cache(8, 32, 1, 1, d, dtype, FAKE, FAKE, FAKE, FAKE)
    b = fox.fox_batch(1, 32767 * Rt, tiles - 2, 0, FAKE, FAKE, FAKE, None)
    assert L.fox_decode(ctypes.byref(c), ctypes.byref(b), 32767 * Rt, FAKE, 128, 0.0, 0, FAKE, FAKE, FAKE, 1 << 50, None) == 2


def test_the_rule_against_plain_numbers(tmp_path):
    src, so = tmp_path / "h.cpp", tmp_path / "h.so"
    src.write_text('#include "fox_paged.h"\nextern "C" int t_fits(long long m, int w, int n) { return fox::line_fits(m, w, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", fbuild.CSRC, str(src), "-o", str(so)], check=True)
    fits = ctypes.CDLL(str(so)).t_fits
    fits.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    for workers, warps in ((608, 4), (1216, 8), (1216, 4), (7, 1)):
        for most in (0, 1, workers, 10**6, INT_MAX // 2, INT_MAX - workers - 1, INT_MAX, 2**31, 2**40, 2**62):
            each = -(-most // workers)
            top = max(most + warps * each, workers * each + each)
            assert not fits(most, workers, warps) or top <= INT_MAX
            assert fits(most, workers, warps) or top + workers + each > INT_MAX


def test_appends_of_more_blocks_than_a_grid_has_are_refused(L):
    """The gates' blocks: a sequence, a page of its most new tokens, 32 heads."""
    c = fox.fox_cache(8, 16, 1024, 1, 64, 0, FAKE, FAKE, FAKE, FAKE)
    for most, status in ((1 << 20, 2), (1 << 16, 3)):  # the second fits, and comes to its missing workspace
        b = fox.fox_batch(2048, most, 1 << 20, 0, FAKE, FAKE, FAKE, None)
        assert L.fox_cache_append(ctypes.byref(c), ctypes.byref(b), (1 << 20) - 1, FAKE, 64, FAKE, 64, FAKE, 1024, None, None,
                                  256, None) == status
