"""Batches whose sequences bring very different counts of new tokens, without a GPU: how much workspace they take, and
the numbers of their items."""
import ctypes
import random
import subprocess

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def workspace(L, B, rows, max_new, H=32, Hkv=8, d=128, dtype=0, stride=512, cu=FAKE):
    c = fox.fox_cache(8, 64, H, Hkv, d, dtype, FAKE, FAKE, FAKE, FAKE)
    b = fox.fox_batch(B, max_new, stride, 0, cu, FAKE, FAKE, None)
    return L.fox_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), rows)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,most", [(64, 16384), (256, 2048), (2048, 4096), (5, 300)])
def test_one_prompt_among_single_tokens(L, B, most, dtype):
    """The partial results that the rows can have: one of every row, a tile's rest a sequence, a tile a worker."""
    rows = most + B - 1
    size = workspace(L, B, rows, most, dtype=dtype)
    Rt = 16 if dtype == 0 else 8
    assert 0 < size <= 1.01 * ((rows * 32 + B * 8 * Rt + 608 * Rt) * (128 + 2) * 4 + 2 * 16384)


def test_equal_counts_take_no_more_than_before(L):
    """Slots of an item each and one a worker: the sizes that uniform batches had."""
    for B, n, G, Rt, Rs, RT in ((64, 1, 4, 8, 4, 1), (16, 4, 4, 16, 16, 1), (3, 7, 4, 16, 16, 2), (2048, 1, 4, 8, 4, 1)):
        slots = 608 + B * 8 * RT
        up = lambda x: -(-x // 256) * 256  # noqa: E731
        want = up(up(up(16384 + 4 * (B + 1)) + slots * Rs * 8) + slots * Rs * 128 * 4)
        assert workspace(L, B, B * n, 1, cu=None) == want


def test_a_mixed_batch_that_fits_by_its_rows_is_taken(L):
    """Twice 2^31 key tiles for the longest sequence's rows in every sequence, far fewer for the rows there are."""
    assert workspace(L, 64, 16384 + 63, 16384, stride=1024) > 0
    assert workspace(L, 64, 64 * 16384, 16384, stride=1024) == 0


def test_numbers_of_items_do_not_meet(tmp_path):
    src, so = tmp_path / "h.cpp", tmp_path / "h.so"
    src.write_text("""#include "fox_paged.h"
// out: items of a key head, whether by rows, then the first number of each sequence
extern "C" void t_items(int rows, int B, int Gp, int sh, int row_tiles, const int* row0, int* out) {
  fox::PagedArgs a = {};
  a.rows = rows; a.B = B;
  long long items;
  const fox::Numbering x = fox::numbering(a, Gp, sh, row_tiles, &items);
  out[0] = items == x.items ? x.items : -1; out[1] = x.by_rows();
  for (int b = 0; b < B; ++b) out[2 + b] = fox::first_item(x, b, row0[b]);
}
extern "C" int t_pad(int G, int Rt) { return fox::padded_group(G, Rt); }
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", fbuild.CSRC, str(src), "-o", str(so)], check=True)
    h = ctypes.CDLL(str(so))
    seen = set()
    rng = random.Random(5)
    for _ in range(400):
        sh, G, B = rng.choice([0, 2, 3, 4]), rng.choice([1, 2, 3, 5, 7, 8, 16, 20, 40]), rng.randint(1, 40)
        Rt = 1 << sh
        Gp = h.t_pad(G, Rt)
        new = [rng.choice([0, 1, 1, 1, 2, rng.randint(0, 300)]) for _ in range(B)]
        # rows that no sequence has, before and between them, are left out
        row0, row = [], rng.randint(0, 3)
        for n in new:
            row0.append(row)
            row += n
        out, end = (ctypes.c_int * (B + 2))(), 0
        most = -(-max(new) * Gp // Rt)
        h.t_items(row + rng.randint(0, 5), B, Gp, sh, max(most, 1), (ctypes.c_int * B)(*row0), out)
        for b in range(B):
            assert out[2 + b] >= end
            end = out[2 + b] + -(-new[b] * Gp // Rt)
        assert end <= out[0] <= B * max(most, 1)
        seen.add(out[1])
    assert seen == {0, 1}
