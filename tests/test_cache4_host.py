"""The 4-bit cache and the pages without a GPU: host refusals of the C ABI, and the 4-bit form's arithmetic and layout, compiled as
plain C++ and compared with a plain restatement (fourtest.py)."""
import ctypes
import os
import subprocess

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or has nothing to do


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def make(cls, base, kw):
    return cls(*[{**base, **kw}[n] for n, _ in cls._fields_])


def _cache(**kw):
    return make(fox.fox_cache4, dict(num_pages=8, page_size=64, H=8, Hkv=2, d=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, g=FAKE, gbase=FAKE,
                                     g_low=None), kw)


def _batch(**kw):
    return make(fox.fox_batch, dict(B=2, max_new=1, table_stride=4, prefix_len=0, cu_new=None, lens=FAKE, table=FAKE, prefix_table=None), kw)


def _decode(L, c=None, s=None, rows=2, q=FAKE, qs=1024, scale=0.0, bj=0, o=1 << 32, lse=1 << 33, ws=FAKE, nbytes=1 << 40):
    return L.fox_cache4_decode(ctypes.byref(c or _cache()), ctypes.byref(s or _batch()), rows, q, qs, scale, bj, o, lse, ws, nbytes, None)


def _append(L, c=None, s=None, rows=2, k=FAKE, ks=256, v=FAKE, vs=256, z=FAKE, zs=8, rot=None, ws=FAKE, nbytes=256):
    return L.fox_cache4_append(ctypes.byref(c or _cache()), ctypes.byref(s or _batch()), rows, k, ks, v, vs, z, zs,
                               None if rot is None else ctypes.byref(rot), ws, nbytes, None)


def _read(L, c=None, s=None, rows=2, k=FAKE, ks=256, v=1 << 32, vs=256, ws=FAKE, nbytes=256):
    return L.fox_cache4_read(ctypes.byref(c or _cache()), ctypes.byref(s or _batch()), rows, k, ks, v, vs, ws, nbytes, None)


def _copy(L, c=None, pairs=FAKE, n=2, ws=FAKE, nbytes=256):
    return L.fox_cache4_copy(ctypes.byref(c or _cache()), pairs, n, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(H=9), 1), (dict(d=0), 1), (dict(d=96), 2), (dict(page_size=48), 2),
    (dict(page_size=256), 2), (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=FAKE + 4), 1),
    (dict(vs=FAKE + 8), 1), (dict(g=None), 1), (dict(gbase=FAKE + 4), 1)])
def test_bad_caches_are_refused(L, kw, status):
    for call in (_decode, _append, _read, _copy):
        assert call(L, _cache(**kw)) == status


def test_more_tokens_of_a_head_than_32_bits_count_are_refused(L):
    for call in (_decode, _append, _read, _copy):
        assert call(L, _cache(num_pages=1 << 26, page_size=64, Hkv=1)) == 2
        assert call(L, _cache(num_pages=(1 << 26) - 1, page_size=64, Hkv=1), ws=None) == 3  # on to the next check


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(B=2049), 2), (dict(table_stride=0), 1), (dict(prefix_len=-1), 1), (dict(prefix_len=5), 1), (dict(lens=None), 1),
    (dict(lens=FAKE + 2), 1), (dict(table=None), 1), (dict(cu_new=FAKE, max_new=0), 1), (dict(cu_new=FAKE + 1), 1),
    (dict(table_stride=1 << 30), 2), (dict(B=3), 1)])
def test_bad_batches_are_refused(L, kw, status):
    for call in (_decode, _append, _read):
        assert call(L, s=_batch(**kw)) == status


def test_bad_rows_and_workspaces_are_refused(L):
    for call in (_decode, _append, _read):
        assert call(L, rows=-2) == 1 and call(L, ws=None) == 3 and call(L, ws=FAKE + 64) == 3 and call(L, nbytes=255) == 3
    assert _decode(L, q=FAKE + 8) == 1 and _decode(L, qs=1023) == 1 and _decode(L, qs=1028) == 1 and _decode(L, o=None) == 1
    assert _decode(L, scale=float("nan")) == 1 and _decode(L, bj=2) == 1 and _decode(L, o=FAKE) == 1 and _decode(L, lse=FAKE) == 1
    need = L.fox_cache4_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(_batch()), 2)
    assert need >= fox.FOX_CACHE_ZERO_BYTES and _decode(L, nbytes=need - 1) == 3
    assert _append(L, k=FAKE + 2) == 1 and _append(L, ks=255) == 1 and _append(L, z=None) == 1 and _append(L, zs=7) == 1
    assert _append(L, _cache(g_low=FAKE + 2)) == 1
    rot = fox.fox_rotary(FAKE, FAKE, 100, 24, 0, None, 0, None)
    assert _append(L, rot=rot) == 2
    rot = fox.fox_rotary(FAKE, FAKE, 100, 64, 0, FAKE, 1024, FAKE + 16)  # over q
    assert _append(L, rot=rot) == 1
    assert _read(L, k=None) == 1 and _read(L, v=FAKE + 8) == 1 and _read(L, ks=252) == 1 and _read(L, v=FAKE + 512) == 1  # over k
    for at in (0, 16, 496, 512, 1536, 2048 - 496):  # rows of 512 bytes, 2048 apart, in each other's
        if at in (512, 1536):
            continue
        assert _read(L, ks=1024, vs=1024, v=FAKE + at) == 1
    assert _read(L, ks=1024, vs=1024, v=FAKE + 512, ws=None) == 3 and _read(L, ks=1024, vs=1024, v=FAKE + 1536, ws=None) == 3  # between them
    assert _copy(L, n=-1) == 1 and _copy(L, pairs=None) == 1 and _copy(L, pairs=FAKE + 4) == 1 and _copy(L, nbytes=255) == 3
    assert _copy(L, n=0x7fffffff) == 2 and _copy(L, n=0, pairs=None, ws=None) == 0
    c2 = fox.fox_cache(8, 64, 8, 2, 128, 0, FAKE, FAKE, FAKE, FAKE)
    assert L.fox_cache_copy(ctypes.byref(c2), FAKE + 8, FAKE, 1, FAKE, 256, None) == 1  # g_low
    assert L.fox_cache_copy(ctypes.byref(c2), None, FAKE, 1, None, 256, None) == 3
    assert L.fox_cache_copy(None, None, FAKE, 1, FAKE, 256, None) == 1


def test_null_arguments_are_refused(L):
    b, c = ctypes.byref(_batch()), ctypes.byref(_cache())
    assert L.fox_cache4_decode(None, b, 2, FAKE, 1024, 0.0, 0, 1 << 32, 1 << 33, FAKE, 1 << 40, None) == 1
    assert L.fox_cache4_decode(c, None, 2, FAKE, 1024, 0.0, 0, 1 << 32, 1 << 33, FAKE, 1 << 40, None) == 1
    assert L.fox_cache4_append(None, b, 2, FAKE, 256, FAKE, 256, FAKE, 8, None, FAKE, 256, None) == 1
    assert L.fox_cache4_read(None, b, 2, FAKE, 256, 1 << 32, 256, FAKE, 256, None) == 1
    assert L.fox_cache4_copy(None, FAKE, 2, FAKE, 256, None) == 1
    assert L.fox_cache4_workspace_bytes(None, b, 2) == 0 and L.fox_cache4_workspace_bytes(c, None, 2) == 0


def test_nothing_to_do_is_ok(L):
    assert _decode(L, s=_batch(B=0), rows=0, q=None, ws=None) == 0 and _append(L, rows=0, k=None, ws=None) == 0
    assert _read(L, rows=0, k=None, v=None, ws=None) == 0


def test_more_work_than_ints_count_is_refused(L):
    big = _batch(B=2048, table_stride=1 << 21)
    assert L.fox_cache4_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(big), 2048) == 0
    assert _decode(L, s=big, rows=2048) == 2


def test_the_extension_passes_what_ctypes_passes(L):
    """_foxcall's calls of the 4-bit cache: the statuses of the same calls by ctypes, whatever argument is bad."""
    from forget_gated_softmax_gb300 import _foxcall

    c, b = _cache(), _batch()
    at = ctypes.addressof(c), ctypes.addressof(b)
    far = 1 << 33
    decode = [*at, 2, FAKE, 1024, 0.0, 0, 1 << 32, far, FAKE, 16, 0]
    append = [*at, 2, FAKE, 256, FAKE, 256, FAKE, 8, FAKE, 16, 0]
    read = [*at, 2, FAKE, 256, 1 << 32, 256, FAKE, 16, 0]
    bad = {2: -1, 3: FAKE + 1, 4: 3, 5: FAKE + 1}
    for name, good in (("decode4", decode), ("append4", append), ("read4", read)):
        for i, x in [(None, None), *bad.items()]:
            if name == "decode4" and i == 5:
                x = float("nan")
            a = list(good) if i is None else [x if j == i else y for j, y in enumerate(good)]
            got = getattr(_foxcall, name)(*a)
            assert got == getattr(fox._CtypesCall, name)(*a) != 0, (name, i)  # at the least the workspace is too small
        with pytest.raises(TypeError):
            getattr(_foxcall, name)(*good[:-1])


# ---- pages ----


def _pages(**kw):
    return make(fox.fox_pages, dict(num_pages=100, page_size=16, B=4, table_stride=8, prefix_len=0, refs=1 << 20, lens=2 << 20, table=3 << 20,
                                    prefix_table=None), kw)


OUT = dict(refs=11 << 20, lens=12 << 20, table=13 << 20)


def _step(L, a=None, b=None, parent=21 << 20, add=22 << 20, copies=23 << 20, ws=FAKE, nbytes=1 << 40):
    return L.fox_pages_step(ctypes.byref(a or _pages()), ctypes.byref(b or _pages(**OUT)), parent, add, copies, ws, nbytes, None)


def _compact(L, a=None, b=None, map=21 << 20, moves=22 << 20, n=10, used=23 << 20, ws=FAKE, nbytes=1 << 40):
    return L.fox_pages_compact(ctypes.byref(a or _pages()), ctypes.byref(b or _pages(**OUT)), map, moves, n, used, ws, nbytes, None)


def test_bad_pages_are_refused(L):
    for kw, status in [(dict(num_pages=0), 1), (dict(num_pages=(1 << 24) + 1), 2), (dict(page_size=24), 2), (dict(B=-1), 1), (dict(B=2049), 2),
                       (dict(table_stride=0), 1), (dict(prefix_len=-1), 1), (dict(table_stride=1 << 28), 2), (dict(refs=None), 1),
                       (dict(refs=(1 << 20) + 2), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(B=2048, table_stride=1 << 20), 2)]:
        for call in (_step, _compact):
            assert call(L, _pages(**kw), _pages(**{**kw, **{n: v for n, v in OUT.items() if n not in kw}})) == status, kw
        assert call(L, None, _pages(**{**OUT, **kw})) != 0 or kw in (dict(lens=None),)
    for kw in (dict(num_pages=101), dict(page_size=32), dict(table_stride=9), dict(prefix_len=4, prefix_table=FAKE)):
        assert _step(L, b=_pages(**{**OUT, **kw})) == 1 and _compact(L, b=_pages(**{**OUT, **kw})) == 1
        assert L.fox_pages_workspace_bytes(ctypes.byref(_pages()), ctypes.byref(_pages(**kw))) == 0
    assert _step(L, b=_pages(B=5, **OUT), parent=None) == 1 and _compact(L, b=_pages(B=5, **OUT)) == 1
    assert _step(L, add=None) == 1 and _step(L, copies=None) == 1 and _step(L, parent=(21 << 20) + 1) == 1
    assert _compact(L, map=None) == 1 and _compact(L, moves=None) == 1 and _compact(L, moves=(22 << 20) + 4) == 1 and _compact(L, used=None) == 1
    assert _compact(L, n=-1) == 1
    assert _compact(L, _pages(prefix_len=4), _pages(prefix_len=4, **OUT)) == 1
    need = L.fox_pages_workspace_bytes(ctypes.byref(_pages()), ctypes.byref(_pages(**OUT)))
    assert need >= fox.FOX_CACHE_ZERO_BYTES
    for call in (_step, _compact):
        assert call(L, ws=None) == 3 and call(L, ws=FAKE + 64) == 3 and call(L, nbytes=need - 1) == 3
    assert L.fox_pages_step(None, ctypes.byref(_pages()), None, FAKE, FAKE, FAKE, 1 << 40, None) == 1
    assert L.fox_pages_workspace_bytes(None, ctypes.byref(_pages())) == 0


def test_pages_outputs_over_other_arguments_are_refused(L):
    # with parent nothing may be in place
    for name in ("refs", "lens", "table"):
        assert _step(L, b=_pages(**{**OUT, name: getattr(_pages(), name)})) == 1
        assert _step(L, b=_pages(**{**OUT, name: getattr(_pages(), name) + 8})) == 1
    # and without it only as a whole
    for name in ("refs", "lens", "table"):
        assert _step(L, b=_pages(**{**OUT, name: getattr(_pages(), name) + 4}), parent=None) == 1
    base = _pages()
    for at in (base.refs, base.lens + 4, base.table, OUT["refs"] + 396, OUT["lens"], 22 << 20):
        assert _step(L, copies=at) == 1
    assert _step(L, b=_pages(**{**OUT, "lens": 22 << 20})) == 1 and _step(L, b=_pages(**{**OUT, "table": 21 << 20})) == 1
    for at in (base.refs, base.lens, base.table, OUT["refs"], OUT["table"], 22 << 20, 23 << 20):
        assert _compact(L, map=at) == 1
    assert _compact(L, used=22 << 20) == 1 and _compact(L, moves=base.table) == 1
    assert _compact(L, b=_pages(**{**OUT, "table": base.table + 4})) == 1


# ---- the form, as the kernels compute it ----

SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "fox_four.h"
using namespace fox;
extern "C" {
int scale_byte(float x) { return (int)four_scale_byte(x); }
float scale(int b) { return four_scale((uint32_t)b); }
int code(float x, int b) { return (int)(four_code_bits(x, b ? 1.f / four_scale((uint32_t)b) : 0.f) - kFourNone); }
unsigned order(unsigned w) { return four_k_order(w); }
long long place(int what, int Hkv, int S, int d, int page, int h, int slot, int b, int t) {
  PagedArgs a = {};
  a.Hkv = Hkv; a.page_size = S; a.d = d;
  const int nb = d / kFourBlock;
  if (what == 0) return (long long)four_row(a, page, h, slot) + four_k_word(b, t, nb);
  if (what == 1) return (long long)four_row(a, page, h, slot) + four_v_word(b, t, slot, nb);
  if (what == 2) return (long long)four_scale_row(a, page, h, slot) + b;
  return (long long)four_scale_row(a, page, h, slot & ~15) + four_v_scale(b, slot, nb);
}
}
"""


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    d = tmp_path_factory.mktemp("form")
    (d / "form.cpp").write_text(SOURCE)
    so = str(d / "form.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I", fbuild.CSRC, str(d / "form.cpp"), "-o", so],
                   check=True)
    F = ctypes.CDLL(so)
    F.scale_byte.argtypes, F.scale.restype, F.code.argtypes = [ctypes.c_float], ctypes.c_float, [ctypes.c_float, ctypes.c_int]
    F.order.argtypes = [ctypes.c_uint]
    F.order.restype = ctypes.c_uint
    F.place.restype = ctypes.c_longlong
    return F


def test_scales(form):
    """Every positive bf16: the byte of the least scale that holds it, by search."""
    import fourtest

    for b, s in enumerate(fourtest.SCALES):
        assert form.scale(b) == s
    x = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    want = torch.searchsorted(7 * torch.tensor(fourtest.SCALES, dtype=torch.float64), x).clamp(max=247)
    got = [form.scale_byte(v) for v in x.tolist()]
    assert got == want.tolist()
    assert form.scale_byte(float("inf")) == 247


def test_codes(form):
    """Every bf16 that a block of each scale may hold, halves among them."""
    import fourtest

    x = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    for b in list(range(0, 12)) + [57, 64, 100, 101, 102, 103, 150, 246, 247]:
        s = fourtest.SCALES[b]
        y = x[(x <= 7 * s) & (x >= s / 300)]
        want = torch.floor(y / s + 0.5) if s else y * 0
        if s:  # the quotient in 64 bits is not a half unless it is one
            assert ((y / s + 0.5 - want).abs() > 2**-40).logical_or(y == (want - 0.5) * s).all()
        for v, u in zip(y.tolist(), want.tolist()):
            assert form.code(v, b) == 8 + u and form.code(-v, b) == 8 - u, (v, b)


@pytest.mark.parametrize("d,S,Hkv", [(64, 16, 1), (128, 16, 3), (64, 128, 2), (128, 64, 8)])
def test_layout(form, d, S, Hkv):
    """The places of the kernels' words and scales, and the order of a word's nibbles, against the places of the bits."""
    import fourtest

    gen = torch.Generator().manual_seed(1)
    for slot in range(S):
        u = torch.randint(-7, 8, (1, 1, d), generator=gen)
        rows = {0: fourtest.row_bytes(u, fourtest.k_bits(d)), 1: fourtest.row_bytes(u, fourtest.v_bits(d, slot))}
        for what, row in rows.items():
            row = bytes(row.flatten().tolist())
            for b in range(d // 32):
                for t in range(4):
                    code = 0
                    for e in range(8):
                        code |= (int(u[0, 0, 32 * b + 8 * t + e]) + 8) << (4 * e)
                    base = ((5 * Hkv + Hkv - 1) * S + slot) * (d // 2)
                    at = form.place(what, Hkv, S, d, 5, Hkv - 1, slot, b, t) - base
                    assert 0 <= at <= d // 2 - 4 and at % 4 == 0
                    word = int.from_bytes(row[at : at + 4], "little")
                    assert word == (code if what else form.order(code))
        for b in range(d // 32):
            base = (5 * Hkv + Hkv - 1) * S * (d // 32)
            assert form.place(2, Hkv, S, d, 5, Hkv - 1, slot, b, 0) == base + slot * (d // 32) + b
            assert form.place(3, Hkv, S, d, 5, Hkv - 1, slot, b, 0) == base + fourtest.v_scale_place(slot, b, d // 32)
    # eight tokens' words of one block lie in different banks, as one ldmatrix reads them
    for s0 in range(0, S, 8):
        for b in range(d // 32):
            at = [form.place(1, 1, S, d, 0, 0, s0 + i, b, 0) % 128 // 16 for i in range(8)]
            assert sorted(at) == list(range(8))
