"""A workspace that is not on the cache's device is refused before anything runs."""
import pytest

torch = pytest.importorskip("torch")

import forget_gated_softmax_gb300 as fox  # noqa: E402


class Fake:
    """What the binding asks of a tensor, on a device of the test's choosing; no memory behind it."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device_index

    def stride(self):
        s, out = 1, []
        for n in reversed(self.shape):
            out.insert(0, s)
            s *= n
        return tuple(out)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("the call went on")

    def numel(self):
        return 1 << 30


@pytest.mark.parametrize("device", [-1, 1])
def test_refused(monkeypatch, device):
    cache, batch = fox.Cache(), fox.Batch()
    cache.H = cache.Hkv = 4
    cache.d, cache.page_size, cache.index, cache.dtype = 64, 16, 0, torch.bfloat16
    cache.device = batch.device = torch.device("cuda", 0)
    batch.prefix_table, cache.g_low = None, None
    monkeypatch.setattr(fox, "_current_device", lambda: 0)
    row, z = (lambda: Fake((2, 4, 64), torch.bfloat16, 0)), Fake((2, 4), torch.float32, 0)
    ws = Fake((1 << 30,), torch.uint8, device)
    with pytest.raises(ValueError, match="ws is not on"):
        fox.fox_decode(cache, batch, row(), o=row(), lse=z, ws=ws)
    with pytest.raises(ValueError, match="ws is not on"):
        fox.fox_cache_append(cache, batch, row(), row(), z, ws=ws)
