"""The gates' running sums in the paged cache, where their rounding shows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    return fox


def Case(*a, **kw):
    from cachetest import Case

    return Case(*a, **kw)


@pytest.mark.parametrize("S,n", [(16, n) for n in range(2, 17)] + [(64, n) for n in (5, 9, 20, 33, 50, 64)] + [(128, 127)])
def test_a_page_begins_at_the_end_of_the_one_before(fox, S, n):
    """One call over a page's end, at every place in it: the next page's base is the base and the last sum that the page
    before holds, bit for bit, as a later call would find them."""
    own = [S * (1 + b % 2) + m for b, m in enumerate(m for m in range(1, n) for _ in range(2))]
    c = Case(own, [n] * len(own), 5, 1, 64, S, uniform=True, seed=n, z_mean=0.0)
    c.put(upto_new=False)
    k, v, z = c.new_rows()
    fox.fox_cache_append(c.cache(fox), c.batch(fox), k, v, z)
    last = torch.tensor([(x - 1) // S for x in own], device="cuda")
    rows = torch.arange(len(own), device="cuda")
    page, before = c.table[rows, last].long(), c.table[rows, last - 1].long()
    sums = c.gbase[before].double().sum(-1) + c.g[before, :, S - 1].double()
    high = sums.float()
    assert not torch.isnan(sums).any()
    assert torch.equal(c.gbase[page, :, 0], high)
    assert torch.equal(c.gbase[page, :, 1], (sums - high.double()).float())
