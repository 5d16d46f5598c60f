"""Page ids outside the pool, in the tables of a decode: reported, read as page 0, and nothing else."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FOX_OK, FOX_ERR_DEVICE = 0, 6


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("B,P,S,new", [(3, 100, 16, 1), (40, 5003, 16, 1), (40, 6000, 64, 2), (4, 70, 32, 9)])
def test_bad_pages_read_as_page_0(B, P, S, new, where, dtype):
    """The same bits as with 0 in the table's place, whether the prefix is walked or (bf16, 40 sequences) shared."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox
    from cachetest import Case

    got = []
    for bad in (True, False):
        c = Case([3 * S + 5] * B, [new] * B, 4, 1, 128, S, dtype=dtype, uniform=True, prefix=P, seed=6)
        c.put()
        for t in (c.k, c.v, c.g, c.gbase):
            t.nan_to_num_(0.0)
        if where == "prefix":
            c.ptable[1], c.ptable[2] = (c.k.shape[0], -1) if bad else (0, 0)
        else:
            c.table[0, 1], c.table[B - 1, 2] = (2**31 - 1, -(2**31)) if bad else (0, 0)
        cache, batch = c.cache(fox), c.batch(fox)
        before = [t.clone() for t in (c.k, c.v, c.g, c.gbase, c.q, c.lens, c.table, c.ptable)]
        ws = fox.cache_workspace(cache, batch, c.rows)
        ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF
        fox.trace_begin()
        o, lse = fox.fox_decode(cache, batch, c.q, ws=ws)
        assert ("prefix" in [k for k, _ in fox.trace_end()]) == (B == 40 and dtype == "bf16")
        assert fox.fox_check_error(ws) == (FOX_ERR_DEVICE if bad else FOX_OK)
        assert fox.fox_check_error(ws) == FOX_OK
        for x, y in zip(before, (c.k, c.v, c.g, c.gbase, c.q, c.lens, c.table, c.ptable)):
            assert torch.equal(bits(x), bits(y))
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        got.append((bits(o), bits(lse)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
