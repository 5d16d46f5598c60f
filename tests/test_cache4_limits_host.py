"""The 4-bit cache's sizes near the ends of 32 bits, without a GPU."""
import ctypes

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def test_row_tiles_of_all_sequences_pass_32_bits(L):
    """2048 sequences of which one may bring all 2^20 rows: 2^20 row tiles each are 2^31 and more of them. The prefix is shared out all the same,
    whatever max_new says beyond that: the rows, and so the workspace, are the same."""
    cache = fox.fox_cache4(64, 64, 32, 1, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None)
    need = []
    for max_new in ((1 << 19) - 1, 1 << 19, (1 << 19) + 1, (1 << 20) - 1, 1 << 20):
        batch = fox.fox_batch(B=2048, max_new=max_new, table_stride=1, prefix_len=2000, cu_new=FAKE, lens=FAKE, table=FAKE, prefix_table=FAKE)
        need.append(L.fox_cache4_workspace_bytes(ctypes.byref(cache), ctypes.byref(batch), 1 << 20))
    assert need[0] > 0 and len(set(need)) == 1
