"""The gates' low parts without a GPU: what the C ABI, the short way from Python and the binding refuse."""
import ctypes

import pytest

import forget_gated_softmax_gb300 as fox
from forget_gated_softmax_gb300 import build as fbuild

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fox.lib()


def handles():
    c = fox.fox_cache(8, 64, 8, 2, 128, 0, FAKE, FAKE, FAKE, FAKE)
    return c, fox.fox_batch(2, 1, 4, 0, None, FAKE, FAKE, None)


def test_a_misaligned_low_part_is_refused(L):
    c, b = handles()
    call = lambda low, ws=FAKE: L.fox_cache_append_low(  # noqa: E731
        ctypes.byref(c), ctypes.byref(b), 2, FAKE, 256, FAKE, 256, FAKE, 8, None, low, ws, 256, None)
    assert call(FAKE + 2) == 1
    assert call(FAKE, ws=None) == 3 and call(None, ws=None) == 3  # the low part is none of its faults


def test_the_short_way_passes_the_low_part(L):
    from forget_gated_softmax_gb300 import _foxcall

    c, b = handles()
    plain = [ctypes.addressof(c), ctypes.addressof(b), 2, FAKE, 256, FAKE, 256, FAKE, 8, FAKE, 256, 0]
    turned = [*plain, FAKE, FAKE, 100, 64, 0, FAKE, 1024, 1 << 30]
    for a in (plain, turned):
        assert _foxcall.append(*a, FAKE + 2) == 1
        a[9] = 0
        assert _foxcall.append(*a, FAKE) == 3 and _foxcall.append(*a, 0) == 3
    with pytest.raises(TypeError):
        _foxcall.append(*plain, 0, 0)


def test_make_cache_refuses_other_low_parts():
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    g, gb = torch.zeros(4, 4, 16), torch.zeros(4, 4, 2)
    with pytest.raises(ValueError, match="g_low"):
        fox.make_cache(k, k.clone(), g, gb, g[:3])
    with pytest.raises(TypeError, match="g_low"):
        fox.make_cache(k, k.clone(), g, gb, g.double())
