"""The paged cache without a GPU: host refusals of the C ABI, and the index arithmetic that decides
every read and write of the pool, compiled as plain C++ and compared with a plain restatement."""
import ctypes
import os
import random
import subprocess

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or has nothing to do


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def _cache(**kw):
    f = dict(num_pages=8, page_size=64, H=8, Hkv=2, d=128, dtype=0, k=FAKE, v=FAKE, g=FAKE, gbase=FAKE)
    f.update(kw)
    return fox.fox_cache(*[f[n] for n, _ in fox.fox_cache._fields_])


def _batch(**kw):
    f = dict(B=2, max_new=1, table_stride=4, prefix_len=0, cu_new=None, lens=FAKE, table=FAKE, prefix_table=None)
    f.update(kw)
    return fox.fox_batch(*[f[n] for n, _ in fox.fox_batch._fields_])


def _decode(L, c=None, s=None, rows=2, q=FAKE, qs=1024, scale=0.0, bj=0, o=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40):
    return L.fox_decode(ctypes.byref(c or _cache()), ctypes.byref(s or _batch()), rows, q, qs, scale, bj, o, lse, ws,
                        nbytes, None)


def _append(L, c=None, s=None, rows=2, k=FAKE, ks=256, v=FAKE, vs=256, z=FAKE, zs=8, rot=None, ws=FAKE, nbytes=256):
    return L.fox_cache_append(ctypes.byref(c or _cache()), ctypes.byref(s or _batch()), rows, k, ks, v, vs, z, zs,
                              None if rot is None else ctypes.byref(rot), ws, nbytes, None)


BAD_CACHE = [
    (dict(num_pages=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(H=9), 1), (dict(dtype=5), 1), (dict(d=0), 1),
    (dict(d=96), 2), (dict(page_size=48), 2), (dict(page_size=0), 2), (dict(page_size=256), 2),
    (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(g=None), 1), (dict(gbase=FAKE + 4), 1),
]
BAD_BATCH = [
    (dict(B=-1), 1), (dict(B=2049), 2), (dict(table_stride=0), 1), (dict(prefix_len=-1), 1),
    (dict(prefix_len=5), 1), (dict(lens=None), 1), (dict(lens=FAKE + 2), 1), (dict(table=None), 1),
    (dict(cu_new=FAKE, max_new=0), 1), (dict(cu_new=FAKE + 1), 1), (dict(table_stride=1 << 30), 2),
    (dict(B=3), 1),  # two rows do not go around three sequences
]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches_are_refused(L, kw, status):
    assert _decode(L, _cache(**kw)) == status
    assert _append(L, _cache(**kw)) == status


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_bad_batches_are_refused(L, kw, status):
    assert _decode(L, s=_batch(**kw)) == status
    assert _append(L, s=_batch(**kw)) == status


def test_bad_rows_scales_and_workspaces_are_refused(L):
    assert _decode(L, rows=-2) == 1 and _append(L, rows=-2) == 1
    assert _decode(L, q=None) == 1 and _decode(L, q=FAKE + 8) == 1
    assert _decode(L, qs=1023) == 1 and _decode(L, qs=1028) == 1  # shorter than a row; no 16-byte multiple
    assert _decode(L, o=None) == 1 and _decode(L, lse=FAKE + 2) == 1
    assert _decode(L, scale=-1.0) == 1 and _decode(L, scale=float("nan")) == 1 and _decode(L, scale=float("inf")) == 1
    assert _decode(L, bj=2) == 1
    need = L.fox_cache_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(_batch()), 2)
    assert need >= 256
    assert _decode(L, nbytes=need - 1) == 3 and _decode(L, ws=None) == 3 and _decode(L, ws=FAKE + 64) == 3
    assert _append(L, k=FAKE + 2) == 1 and _append(L, ks=255) == 1 and _append(L, vs=260) == 1
    assert _append(L, z=None) == 1 and _append(L, zs=7) == 1
    assert _append(L, ws=None) == 3 and _append(L, nbytes=255) == 3
    assert L.fox_decode(None, None, 1, FAKE, 8, 0.0, 0, FAKE, FAKE, FAKE, 256, None) == 1
    assert L.fox_cache_append(ctypes.byref(_cache()), None, 1, FAKE, 8, FAKE, 8, FAKE, 8, None, FAKE, 256, None) == 1


def test_more_work_than_ints_count_is_refused(L):
    big = _batch(B=2048, table_stride=1 << 21)  # 134 million tokens a sequence
    assert L.fox_cache_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(big), 2048) == 0
    assert _decode(L, s=big, rows=2048) == 2
    fits = _batch(B=2048, table_stride=1 << 11)
    assert L.fox_cache_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(fits), 2048) > 0


def test_bad_rotations_are_refused(L):
    def rot(**kw):
        f = dict(cos=FAKE, sin=FAKE, max_pos=100, dim=64, pairs=0, q=None, q_stride=0, q_out=None)
        f.update(kw)
        return fox.fox_rotary(*[f[n] for n, _ in fox.fox_rotary._fields_])

    for kw, status in [(dict(dim=-16), 1), (dict(pairs=2), 1), (dict(max_pos=-1), 1), (dict(dim=24), 2),
                       (dict(dim=144), 2), (dict(cos=None), 1), (dict(sin=FAKE + 4), 1), (dict(q=FAKE, q_stride=1024), 1),
                       (dict(q=FAKE, q_stride=8, q_out=FAKE), 1), (dict(q=FAKE + 2, q_stride=1024, q_out=FAKE), 1)]:
        assert _append(L, rot=rot(**kw)) == status, kw


def test_outputs_over_the_rows_they_are_made_from_are_refused(L):
    row = 8 * 128 * 2
    for o in (FAKE, FAKE + 16, FAKE + 2 * row - 16, FAKE - 2 * row + 16):
        assert _decode(L, q=FAKE, o=o) == 1
        rot = fox.fox_rotary(FAKE, FAKE, 100, 64, 0, FAKE, 1024, o)
        assert _append(L, rot=rot) == 1
    assert _decode(L, q=FAKE, qs=1 << 39, rows=2, o=FAKE + (1 << 38)) == 1  # between rows that lie far apart


def test_nothing_to_do_is_ok(L):
    assert _decode(L, s=_batch(B=0), rows=0, q=None, o=None, lse=None, ws=None, nbytes=0) == 0
    assert _decode(L, rows=0, q=None, ws=None, nbytes=0) == 0
    assert _append(L, s=_batch(B=0), rows=0, k=None, ws=None, nbytes=0) == 0
    assert L.fox_cache_workspace_bytes(ctypes.byref(_cache(d=96)), ctypes.byref(_batch()), 2) == 0
    assert L.fox_cache_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(_batch(B=0)), 0) == fox.FOX_CACHE_ZERO_BYTES


def test_binding_refuses_what_is_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    g, gb = torch.zeros(4, 4, 16), torch.zeros(4, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fox.make_cache(k, k.clone(), g, gb)
    with pytest.raises(ValueError, match="k's shape"):
        fox.make_cache(k, k[:3], g, gb)
    with pytest.raises(ValueError, match="page_size"):
        fox.make_cache(k, k.clone(), g[:, :, :8], gb)
    with pytest.raises(TypeError):
        fox.make_cache(k, k.clone(), g.double(), gb)
    lens, table = torch.ones(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fox.make_batch(lens, table)
    with pytest.raises(ValueError, match="max_new"):
        fox.make_batch(lens, table, cu_new=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        fox.make_batch(lens.long(), table)
    with pytest.raises(ValueError):
        fox.make_batch(lens, table[:1])
    with pytest.raises(ValueError, match="together"):
        fox.make_batch(lens, table, prefix_len=3)


# ---------------------------------------------------------------------------------- index arithmetic

HARNESS = r"""
#include "fox_paged.h"
using namespace fox;
static PagedArgs args(const int* n, const int* cu, const int* lens, const int* table, const int* prefix) {
  PagedArgs a = {};
  a.num_pages = n[0]; a.page_size = n[1]; a.H = n[2]; a.Hkv = n[3]; a.d = n[4]; a.B = n[5]; a.rows = n[6];
  a.max_new = n[7]; a.page_shift = __builtin_ctz(n[1]); a.table_stride = n[8]; a.prefix_len = n[9];
  a.cu = cu; a.lens = lens; a.table = table; a.prefix = prefix;
  return a;
}
extern "C" {
void t_seq(const int* n, const int* cu, const int* lens, int b, int* out) {
  bool bad;
  const SeqInfo s = seq_info(args(n, cu, lens, nullptr, nullptr), b, &bad);
  out[0] = s.row0; out[1] = s.n; out[2] = s.own; out[3] = bad;
}
int t_seq_of_row(const int* n, const int* cu, int i) { return seq_of_row(args(n, cu, nullptr, nullptr, nullptr), i); }
int t_own_page(const int* n, const int* table, int b, int p) { return own_page(args(n, nullptr, nullptr, table, nullptr), b, p); }
int t_prefix_page(const int* n, const int* prefix, int p) { return prefix_page(args(n, nullptr, nullptr, nullptr, prefix), p); }
long long t_kv(const int* n, int page, int h, int s) { return (long long)kv_offset(args(n, nullptr, nullptr, nullptr, nullptr), page, h, s); }
long long t_g(const int* n, int page, int h, int s) { return (long long)g_offset(args(n, nullptr, nullptr, nullptr, nullptr), page, h, s); }
int t_units(const int* n, const int* cu, const int* lens, int b, int Rt, int walk) {
  const PagedArgs a = args(n, cu, lens, nullptr, nullptr);
  bool bad;
  return seq_units(a, seq_info(a, b, &bad), Rt, padded_group(a.H / a.Hkv, Rt), walk);
}
int t_each(int total, int workers) { return units_per_worker(total, workers); }
}
"""


@pytest.fixture(scope="module")
def H(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src, so = d / "h.cpp", d / "h.so"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", fbuild.CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for f in ("t_kv", "t_g"):
        getattr(lib, f).restype = ctypes.c_longlong
    return lib


def _ints(xs):
    return (ctypes.c_int * max(1, len(xs)))(*xs)


def _n(pages=10, S=16, H=4, Hkv=2, d=64, B=1, rows=1, max_new=1, stride=4, prefix=0):
    return _ints([pages, S, H, Hkv, d, B, rows, max_new, stride, prefix])


def _seq(H, n, cu, lens, b):
    out = _ints([0] * 4)
    H.t_seq(n, None if cu is None else _ints(cu), _ints(lens), b, out)
    return list(out)


def test_sequences_that_the_batch_cannot_hold_have_no_rows(H):
    n = _n(B=3, rows=7, max_new=4, prefix=20)  # holds 20 + 4 * 16 tokens
    for cu, lens, b, want in [
        ([0, 2, 3, 7], [22, 84, 0], 0, [0, 2, 2, 0]),
        ([0, 2, 3, 7], [22, 84, 0], 1, [2, 1, 64, 0]),
        ([0, 2, 3, 7], [22, 84, 0], 2, [3, 4, -1, 0]),    # idle: keeps its rows
        ([0, 2, 3, 7], [21, 85, -1], 0, [0, 0, -1, 1]),   # new tokens inside the prefix
        ([0, 2, 3, 7], [21, 85, -1], 1, [0, 0, -1, 1]),   # more than the table holds
        ([0, 2, 3, 7], [21, 85, -1], 2, [0, 0, -1, 1]),
        ([0, 2, 1, 7], [60, 60, 60], 1, [0, 0, -1, 1]),   # falling
        ([0, 2, 3, 8], [60, 60, 60], 2, [0, 0, -1, 1]),   # behind the rows, and more than max_new
        ([-1, 2, 3, 7], [60, 60, 60], 0, [0, 0, -1, 1]),
        ([0, 0, 0, 0], [60, 60, 60], 1, [0, 0, 40, 0]),   # no new tokens
        ([0, 2, 3, 7], [22, 2**31 - 1, 0], 1, [0, 0, -1, 1]),
    ]:
        assert _seq(H, n, cu, lens, b) == want, (cu, lens, b)
    assert _seq(H, _n(B=3, rows=6, max_new=2), None, [5, 6, 1], 1) == [2, 2, 6, 0]
    assert _seq(H, _n(B=3, rows=6, max_new=2), None, [5, 6, 1], 2) == [0, 0, -1, 1]


def test_rows_find_their_sequence_whatever_cu_holds(H):
    rng = random.Random(3)
    for _ in range(200):
        B = rng.randint(1, 9)
        new = [rng.randint(0, 5) for _ in range(B)]
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        rows = cu[-1] + rng.randint(0, 3)
        n = _n(B=B, rows=rows)
        for i in range(rows):
            want = next((b for b in range(B) if cu[b] <= i < cu[b + 1]), -1)
            assert H.t_seq_of_row(n, _ints(cu), i) == want
        junk = [rng.randint(-5, 20) for _ in range(B + 1)]
        for i in range(20):
            assert -1 <= H.t_seq_of_row(n, _ints(junk), i) < B
    for i in range(12):
        assert H.t_seq_of_row(_n(B=4, rows=12), None, i) == i // 3


def test_page_ids_outside_the_pool_are_no_pages(H):
    n = _n(pages=10, S=16, B=2, stride=3)
    table = [3, 9, 10, -1, 0, 2**31 - 1]
    assert [H.t_own_page(n, _ints(table), 0, p) for p in (0, 15, 16, 47)] == [3, 3, 9, -1]
    assert [H.t_own_page(n, _ints(table), 1, p) for p in (0, 16, 31, 32)] == [-1, 0, 0, -1]
    assert [H.t_prefix_page(n, _ints([4, -7]), p) for p in (0, 15, 16)] == [4, 4, -1]


def test_offsets_pass_32_bits(H):
    n = _n(pages=200000, S=128, H=32, Hkv=8, d=128)
    assert H.t_kv(n, 199999, 7, 127) == ((199999 * 8 + 7) * 128 + 127) * 128 > 2**32
    assert H.t_g(n, 199999, 31, 127) == (199999 * 32 + 31) * 128 + 127


@pytest.mark.parametrize("workers", [1, 7, 608, 2432])
def test_work_line_gives_every_pair_of_worker_and_item_its_own_slot(H, workers):
    """The units of all items on one line, cut into equal ranges: each pair's slot (worker + item) is
    its own, and fewer than workers + items are in use."""
    rng = random.Random(workers)
    for _ in range(30):
        B, Hkv, G = rng.randint(1, 12), rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 7, 20])
        new = [rng.randint(0, 9) for _ in range(B)]
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        P, walk = rng.choice([0, 45]), rng.choice([0, 1])
        own = [rng.choice([None, x + rng.randint(0, 1000)]) if x else rng.randint(1, 50) for x in new]
        lens = [0 if y is None else P + y for y in own]
        Rt = rng.choice([8, 16, 32])
        n = _n(H=G * Hkv, Hkv=Hkv, B=B, rows=max(1, cu[-1]), max_new=max(new + [1]), stride=100, prefix=P)
        units = [H.t_units(n, _ints(cu), _ints(lens), b, Rt, walk) for b in range(B)]
        tiles_of = [0 if y is None else -(-y // 32) + (-(-P // 32) if walk else 0) for y in own]
        Gp = G if G <= Rt else -(-G // Rt) * Rt  # a token's rows fill whole row tiles, or lie in one
        rts = [-(-x * Gp // Rt) for x in new]
        assert units == [y * r for y, r in zip(tiles_of, rts)]
        total = sum(units) * Hkv
        each = H.t_each(total, workers)
        assert each * workers >= total and each >= 1
        RTmax, u, slots = -(-max(new + [1]) * Gp // Rt), 0, set()
        for h in range(Hkv):
            for b in range(B):
                for rt in range(rts[b]):
                    tiles, item = tiles_of[b], (h * B + b) * RTmax + rt
                    if not tiles:
                        continue
                    for w in range(u // each, (u + tiles - 1) // each + 1):
                        assert w < workers and (w + item) not in slots
                        slots.add(w + item)
                    u += tiles
        assert u == total
        assert not slots or max(slots) < workers + Hkv * B * RTmax


def test_the_short_way_passes_the_same_arguments(L):
    """_foxcall's append and decode against ctypes: the same statuses, each argument in its place."""
    from forget_gated_softmax_gb300 import _foxcall

    c, s = _cache(), _batch()
    need = L.fox_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(s), 2)
    at = (ctypes.addressof(c), ctypes.addressof(s))
    good = [*at, 2, FAKE, 1024, 0.5, 1, 1 << 30, FAKE, FAKE, need, 0]
    for i, v, status in [(2, -2, 1), (2, 3, 1), (3, 0, 1), (3, FAKE + 8, 1), (4, 1023, 1), (5, -1.0, 1), (5, float("nan"), 1),
                         (6, 2, 1), (7, 0, 1), (7, FAKE + 16, 1), (8, FAKE + 2, 1), (9, FAKE + 64, 3), (10, need - 1, 3)]:
        a = list(good)
        a[i] = v
        assert _foxcall.decode(*a) == status, (i, v)
    good = [*at, 2, FAKE, 256, FAKE, 256, FAKE, 8, FAKE, 256, 0, FAKE, FAKE, 100, 64, 0, FAKE, 1024, 1 << 30]
    for i, v, status in [(2, -2, 1), (3, FAKE + 2, 1), (4, 255, 1), (5, 0, 1), (6, 260, 1), (7, 0, 1), (8, 7, 1), (9, 0, 3),
                         (10, 255, 3), (12, 0, 1), (13, FAKE + 4, 1), (14, -1, 1), (15, 24, 2), (15, -16, 1), (16, 2, 1),
                         (17, FAKE + 2, 1), (18, 8, 1), (19, 0, 1), (19, FAKE + 16, 1)]:
        a = list(good)
        a[i] = v
        assert _foxcall.append(*a) == status, (i, v)
    assert _foxcall.append(*good[:9], 0, 0, 0) == 3
    for bad in ([1], [*good[:11]], ["x"] * 12, [1 << 70] * 12):
        with pytest.raises((TypeError, OverflowError)):
            _foxcall.decode(*bad)
        with pytest.raises((TypeError, OverflowError)):
            _foxcall.append(*bad)
    with pytest.raises(OverflowError):
        _foxcall.decode(*at, 1 << 31, FAKE, 1024, 0.5, 1, 1 << 30, FAKE, FAKE, need, 0)
