"""libfox.so is all that the binding needs: without _foxcall.so every function works, the serving calls by ctypes."""
import ctypes
import os
import subprocess
import sys

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

FAKE = 0x10000  # never dereferenced: every call below fails validation first
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def test_the_library_loads_without_it(L):
    code = (
        "import sys; sys.modules['forget_gated_softmax_gb300._foxcall'] = None\n"
        "import forget_gated_softmax_gb300 as fox\n"
        "assert fox.fox_fwd_workspace_bytes(fox.make_params(1, 256, 2, 64)) > 0\n"
        "assert fox._load_call() is fox._CtypesCall\n"
    )
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


def test_both_ways_give_the_same_statuses(L):
    from forget_gated_softmax_gb300 import _foxcall

    c = fox.fox_cache(8, 64, 8, 2, 128, 0, FAKE, FAKE, FAKE, FAKE)
    b = fox.fox_batch(2, 1, 4, 0, None, FAKE, FAKE, None)
    at = (ctypes.addressof(c), ctypes.addressof(b))
    need = L.fox_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 2)
    decode = [*at, 2, FAKE, 1024, 0.5, 1, 1 << 30, FAKE, FAKE, need, 0]
    plain = [*at, 2, FAKE, 256, FAKE, 256, FAKE, 8, FAKE, 256, 0]
    rot = [FAKE, FAKE, 100, 64, 0, FAKE, 1024, 1 << 30]
    seen = set()
    for name, good in (("decode", decode), ("append", plain), ("append", plain + [FAKE]), ("append", plain + rot),
                       ("append", plain + rot + [FAKE])):
        for i in range(2, len(good)):
            for v in (-1.0,) if isinstance(good[i], float) else (-2, 3, FAKE + 2, FAKE + 64, 0):
                a = list(good)
                a[i] = v
                if name == "append":
                    a[9] = v if i == 9 else 0  # no workspace: nothing runs, whatever else is right
                else:
                    a[10] = min(a[10], need - 1) if i != 10 else 0
                if i == 9 or any(x < 0 for j, x in enumerate(a) if j in (3, 5, 7, 8, 9, 10, 11, 12, 13, 17, 19, 20)):
                    continue  # addresses and sizes are no negative numbers
                want = getattr(_foxcall, name)(*a)
                assert getattr(fox._CtypesCall, name)(*a) == want, (name, i, v)
                assert want or a[2] == 0  # nothing to do
                seen.add(want)
    assert seen >= {1, 2, 3}


def test_the_build_goes_on_without_python_s_headers(L, monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(fbuild, "CALL", str(tmp_path / "_foxcall.so"))
    monkeypatch.setattr(fbuild.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    fbuild._build_call()
    assert not os.path.exists(fbuild.CALL) and "ctypes" in capsys.readouterr().err


@pytest.mark.gpu
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("low", [False, True])
def test_both_ways_give_the_same_results(L, monkeypatch, turned, low):
    torch = pytest.importorskip("torch")
    from cachetest import Case

    got = []
    for way in (fox._load_call(), fox._CtypesCall):
        monkeypatch.setattr(fox, "_call", way)
        c = Case([40, 7], [3, 1], 8, 2, 64, 16, seed=2)
        c.put(upto_new=False)
        for t in (c.k, c.v, c.g, c.gbase):
            t.nan_to_num_(0.0)
        k, v, z = c.new_rows()
        kw = dict(q=c.q, cos=torch.ones(50, 16, device="cuda"), sin=torch.full((50, 16), 0.5, device="cuda")) if turned else {}
        g_low = torch.zeros_like(c.g) if low else None
        cache = fox.make_cache(c.k, c.v, c.g, c.gbase, g_low)
        q = fox.fox_cache_append(cache, c.batch(fox), k, v, z, **kw)
        o, lse = fox.fox_decode(cache, c.batch(fox), c.q)
        got.append([t for t in (c.k, c.v, c.g, c.gbase, g_low, q, o, lse) if t is not None])
    assert len(got[0]) == len(got[1]) == 6 + turned + low
    for a, b in zip(*got):
        assert torch.equal(a, b)
