"""Outputs of the paged-cache calls that lie over their other arguments are refused on the host."""
import ctypes

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

MB = 1 << 20  # arguments a MB apart; never dereferenced: every call below fails validation
ROWS, H, HKV, D = 5, 8, 2, 128


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def handles(dtype):
    c = fox.fox_cache(8, 64, H, HKV, D, dtype, MB, MB, MB, MB)
    return c, fox.fox_batch(ROWS, 1, 4, 0, None, MB, MB, None)


@pytest.mark.parametrize("dtype,es", [(0, 2), (1, 4)])
def test_append(L, dtype, es):
    c, b = handles(dtype)
    row, kv = H * D, HKV * D
    # where each argument lies, its bytes from the first to the last, rows 100 elements (a multiple of 16 bytes) apart
    wide = lambda n: n + 104  # noqa: E731
    args = {"k": (2 * MB, (4 * wide(kv) + kv) * es), "v": (3 * MB, (4 * wide(kv) + kv) * es), "z": (4 * MB, (4 * (H + 3) + H) * 4),
            "q": (5 * MB, (4 * wide(row) + row) * es), "cos": (6 * MB, 100 * 32 * 4), "sin": (7 * MB, 100 * 32 * 4)}
    out = ROWS * row * es

    def call(q_out):
        rot = fox.fox_rotary(args["cos"][0], args["sin"][0], 100, 64, 0, args["q"][0], wide(row), q_out)
        return L.fox_cache_append(ctypes.byref(c), ctypes.byref(b), ROWS, args["k"][0], wide(kv), args["v"][0], wide(kv),
                                  args["z"][0], H + 3, ctypes.byref(rot), MB, 256, None)

    for name, (at, n) in args.items():
        for q_out in (at, at - out + 16, (at + n - 1) // 16 * 16, at + n // 32 * 16):
            assert call(q_out) == 1, (name, q_out - at)


@pytest.mark.parametrize("dtype,es", [(0, 2), (1, 4)])
def test_decode(L, dtype, es):
    c, b = handles(dtype)
    row = H * D
    need = L.fox_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), ROWS)
    out, lse_bytes = ROWS * row * es, ROWS * H * 4

    def call(q, o, lse):
        return L.fox_decode(ctypes.byref(c), ctypes.byref(b), ROWS, q, row + 8, 0.0, 0, o, lse, MB, need, None)

    q, n = 5 * MB, (4 * (row + 8) + row) * es
    for at in (q, q - lse_bytes + 4, q + n - 4, q + n // 8 * 4):
        assert call(q, 8 * MB, at) == 1, at - q
    for at in (q, q - out + 16, (q + n - 1) // 16 * 16):
        assert call(q, at, 8 * MB) == 1, at - q
    for at in (8 * MB, 8 * MB - lse_bytes + 4, 8 * MB + out - 4, 8 * MB + out // 2):
        assert call(q, 8 * MB, at) == 1, at
