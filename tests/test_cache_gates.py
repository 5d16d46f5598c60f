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


def one_at_a_time(fox, cache, c, first=0):
    """Sequence 0's tokens from `first` on, appended by calls of one token each."""
    k, v, z = c.seq[0]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    batch = fox.make_batch(lens, c.table)
    for t in range(first, c.own[0]):
        lens.fill_(t + 1)
        fox.fox_cache_append(cache, batch, k[t : t + 1], v[t : t + 1], z[t : t + 1], ws=ws)
    assert fox.fox_check_error(ws) == 0
    return batch, ws


def sums(cache, table, n, S):
    """Cumulative log gates [n, H] as the cache holds them."""
    t = torch.arange(n, device="cuda")
    page = table[0, t // S].long()
    return cache.gbase[page].double().sum(-1) + cache.g[page, :, t % S].double()


# strong gates and the weak ones behind them, tokens, page
STRONG = [(-1.0e4, 8.0, 127, 128), (-4000.0, 9.0, 128, 128), (-1.0e4, 6.0, 300, 128), (-300.0, 7.0, 200, 64), (-2.0e5, 3.0, 16, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("strong,weak,n,S", STRONG)
def test_weak_gates_behind_a_strong_one_count(fox, strong, weak, n, S, dtype):
    """Token by token: c of the tokens behind the strong gate from the next one on, and attention over them. Each g is
    its sum rounded once, 2^-24 of |g| at most, and log sigmoid is within 8 * 2^-24 of itself, so c_i - c_j is off by
    2 * 2^-24 |g| and 8 * 2^-24 of itself, and a page's base (two fp32, 2^-48) by nothing to speak of. Scores off by d
    move LSE by d and weights by factors within exp(2 d)."""
    from cachetest import log_f

    import foxtest

    H, d = 4, 64
    c = Case([n], [1], H, 2, d, S, dtype=dtype, seed=7)
    z = c.seq[0][2]
    z.fill_(weak)
    z += torch.linspace(0, 0.5, H, device="cuda")
    z[1] = strong
    cache = fox.new_cache(c.k.shape[0], S, H, 2, d, dtype=c.dt)
    for t in (cache.g, cache.gbase, cache.g_low):
        t.fill_(float("nan"))
    batch, ws = one_at_a_time(fox, cache, c)
    want = log_f(z).cumsum(0)
    got = sums(cache, c.table, n, S)
    d_got, d_want = (x[2:] - x[2] for x in (got, want))
    g_most = -strong * 1.001 + 64
    off = (d_got - d_want).abs() - 8 * 2.0**-24 * d_want.abs()
    assert off.max().item() <= 2 * 2.0**-24 * g_most
    o, lse = fox.fox_decode(cache, batch, c.q)
    ro, rl = c.attend()
    delta = 2 * 2.0**-24 * g_most + 8 * 2.0**-24 * d_want.abs().max().item()
    tol_o, tol_l = (foxtest.TOL_O_BF16, foxtest.TOL_LSE_BF16) if dtype == "bf16" else (foxtest.TOL_O_F32, foxtest.TOL_LSE_F32)
    assert (lse.double() - rl).abs().max().item() <= tol_l + delta
    most = c.seq[0][1].double().abs().max().item()
    assert (o.double() - ro).abs().max().item() <= tol_o + 2.1 * delta * 2 * most
    # the same call again writes the same values
    before = [x.clone() for x in (cache.g, cache.g_low, cache.gbase)]
    k, v, z = (x[n - 1 :] for x in c.seq[0])
    fox.fox_cache_append(cache, batch, k, v, z, ws=ws)
    for x, y in zip(before, (cache.g, cache.g_low, cache.gbase)):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))


@pytest.mark.parametrize("what", ["none", "nan", "huge", "small"])
def test_sums_without_their_low_parts(fox, what):
    """A cache without g_low, or one whose g_low holds anything else (here between two calls): each call adds a rounding
    of g, 2^-24 of it; no more."""
    from cachetest import log_f

    n, S, H = 100, 128, 4
    c = Case([n], [1], H, 2, 64, S, seed=8)
    z = c.seq[0][2]
    z.fill_(5.0)
    z[1] = -1000.0
    cache = fox.new_cache(c.k.shape[0], S, H, 2, 64)
    if what == "none":
        cache = fox.make_cache(cache.k, cache.v, cache.g, cache.gbase)
    fill = {"nan": float("nan"), "huge": -1.0e30, "small": 2.0**-14}  # the last less than half a step of g
    k, v, z = c.seq[0]
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    batch = fox.make_batch(lens, c.table)
    for t in range(n):
        lens.fill_(t + 1)
        if what != "none":
            cache.g_low.fill_(fill[what])
        fox.fox_cache_append(cache, batch, k[t : t + 1], v[t : t + 1], z[t : t + 1])
    want, got = log_f(z).cumsum(0), sums(cache, c.table, n, S)
    # a wrong low part of at most half a step comes on top of the rounding
    assert ((got - want).abs() <= (n + 8) * 2.0**-24 * want.abs() * (2 if what == "small" else 1)).all()


@pytest.mark.parametrize("n", [3, 8, 9, 40])
def test_calls_of_several_tokens_go_on_from_the_whole_sum(fox, n):
    """A strong gate, then calls of n tokens over several pages, the last page's end inside a call."""
    from cachetest import log_f

    S, H, own = 64, 4, 1 + 5 * 40
    c = Case([own], [1], H, 2, 64, S, seed=9)
    k, v, z = c.seq[0]
    z.fill_(8.0)
    z[0] = -5000.0
    cache = fox.new_cache(c.k.shape[0], S, H, 2, 64)
    lens, cu = torch.empty(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    batch = fox.make_batch(lens, c.table, cu_new=cu, max_new=n)
    t = 0
    while t < own:
        m = 1 if t == 0 else min(n, own - t)
        lens.fill_(t + m)
        cu[1] = m
        fox.fox_cache_append(cache, batch, k[t : t + m], v[t : t + m], z[t : t + m])
        t += m
    want, got = log_f(z).cumsum(0), sums(cache, c.table, own, S)
    d_got, d_want = (x[1:] - x[1] for x in (got, want))
    # calls of more than 8 tokens sum them apart by a scan: relative to their own sum, 11 roundings
    assert ((d_got - d_want).abs() <= 2 * 2.0**-24 * 5001 + (8 + 11) * 2.0**-24 * d_want.abs()).all()
