"""The decode over the 4-bit cache where its sums need range: small values, small weights, large values beside them. Each case is
one that has a closed form: a first key of weight 1 whose V is 0, and n keys of weight w = 2^-e that agree.

O = n w v / (1 + n w), to be met in relation to itself. Weights and their products with scales come in fp16, at 2^10 times their value
against the first key's at least: w >= 2^-24 keeps 11 bits (a half step of 2^-11 of itself), as does the product with a scale that is brought to
[1, 2), so that O is off by 2^-11 for each of the two, by n sums in fp32 (2^-24 each at most, of terms of one sign: below 2^-11 for n up to 8192)
and by its own rounding, 2^-8 at most: 2^-8 + 3 * 2^-11 of O."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TOL = 2.0**-8 + 3 * 2.0**-11


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    fox.lib()
    return fox


def sink(B, G, Hkv, d, n, e, v, prefix=0, new=1):
    """B sequences of a first key (the prefix's, if there is one) and n others 2^-e of its weight; V [d] of those. Rows of work are
    as many as workers, so that one worker has the first key and most of the others."""
    from fourtest import Case4

    c = Case4([n + (0 if prefix else 1)] * B, [new] * B, G * Hkv, Hkv, d, 64, uniform=True, seed=5, prefix=prefix)
    # K is 0 but in the first key's channel 0
    q0 = torch.zeros(d, device="cuda")
    q0[0] = 1.0
    c.q[:] = q0.bfloat16()
    for k, vv, z in [c.pre, *c.seq]:
        k.zero_()
        vv[:] = v.bfloat16()
        z.fill_(float("inf"))  # no decay
    first = [c.pre] if prefix else c.seq
    for k, vv, z in first:
        k[0, :, 0] = 1.75  # 7 * 0.25: held as it is
        vv[0] = 0.0
    return c, e * 0.6931471805599453 / 1.75


def decode(fox, c, scale):
    c.put()
    cache, batch = c.cache4(fox), c.batch(fox)
    ws = fox.cache4_workspace(cache, batch, c.rows)
    o, lse = fox.fox_cache4_decode(cache, batch, c.q, scale=scale, ws=ws)
    assert fox.fox_check_error(ws) == 0
    return o, lse


def held(c):
    """The last token's V, as it is held: [Hkv, d] in 64 bits."""
    return c.held[0][1][-1]


def check(o, c, n, e, tol=TOL):
    G = c.H // c.Hkv
    want = held(c) * (n * 2.0**-e / (1 + n * 2.0**-e))
    want = want[None, :, None].expand(c.rows, -1, G, -1).reshape(o.shape)
    off = ((o.double() - want).abs() / want.abs())
    assert (off <= tol).all(), off.max().item()


@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (8, 128), (12, 64)])  # tiles of 4, 4, 8 and 16 rows
@pytest.mark.parametrize("size", [1.0, 0.05, 1.0e-3, 2.0**-15, 112.0, 30000.0])
@pytest.mark.parametrize("e", [18, 21, 24])
def test_small_weights_of_values_of_any_size(fox, G, d, size, e):
    n = 1500
    v = torch.full((d,), size, device="cuda")
    c, scale = sink(64, G, 32, d, n, e, v)
    o, _ = decode(fox, c, scale)
    check(o, c, n, e)


@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (12, 64)])
@pytest.mark.parametrize("late", [False, True])
def test_a_large_block_leaves_the_other_channels_alone(fox, G, d, late):
    """One key whose first 32 channels of V are 7000 (and whose weight is 2^-24 like the others'): the other channels lose nothing."""
    n, e = 1500, 24
    v = torch.full((d,), 0.05, device="cuda")
    c, scale = sink(64, G, 32, d, n, e, v)
    for k, vv, z in c.seq:
        vv[n - 40 if late else 3, :, :32] = 7000.0
    o, _ = decode(fox, c, scale)
    assert torch.equal(held(c)[:, 32:], c.held[0][1][n - 40 if late else 3][:, 32:])
    G = c.H // c.Hkv
    want = held(c) * (n * 2.0**-e / (1 + n * 2.0**-e))
    want = want[None, :, None].expand(c.rows, -1, G, -1).reshape(o.shape)
    off = ((o.double() - want).abs() / want.abs())[..., 32:]
    assert (off <= TOL).all(), off.max().item()


def test_sizes_that_change_along_a_sequence(fox):
    """V of 2^-14 first, then of ever larger size, or the other way round: the sums so far are brought to the new size. O is met in relation to
    a mean of |V| by the weights: 2^-8 and 2^-11 for weights, products and scores each (keys of equal weights, 4096 at most)."""
    from fourtest import Case4

    for back in (False, True):
        c = Case4([1200, 70], [1, 3], 8, 2, 128, 32, seed=77)
        for i, (k, v, z) in enumerate(c.seq):
            size = 2.0 ** torch.linspace(-14, 13, v.shape[0], device="cuda")
            c.seq[i] = (k, (v * (size.flip(0) if back else size)[:, None, None]).bfloat16(), z + 6)
        o, _ = decode(fox, c, 0.0)
        ro, _ = c.attend()
        keep = c.held
        c.held = {b: (x[0], x[1].abs()) for b, x in keep.items()}
        mean, _ = c.attend()
        assert ((o.double() - ro).abs() <= 2.0**-8 * ro.abs() + 3 * 2.0**-11 * mean).all()


@pytest.mark.parametrize("walked", [True, False])
def test_small_values_behind_a_prefix(fox, walked):
    """The first key is the prefix's, which is walked, or spread out and shared: the same O."""
    n, e = 1500, 22
    B, P = (64, 40) if walked else (150, 5003)
    v = torch.full((64,), 0.003, device="cuda")
    c, scale = sink(B, 1, 8, 64, n, e, v, prefix=P)
    o, _ = decode(fox, c, scale)
    check(o, c, n + P - 1, e)


@pytest.mark.parametrize("G,d,new", [(1, 128, 3), (4, 64, 2), (4, 128, 3), (8, 64, 5)])  # tiles of 4, 8, 16 and of 16 rows, three a sequence
@pytest.mark.parametrize("size,e", [(1.0e-3, 24), (0.05, 21), (30000.0, 24)])
def test_several_new_tokens(fox, G, d, new, size, e):
    """Row t of a sequence sees new - 1 - t keys fewer than its last one."""
    n = 1500
    c, scale = sink(64, G, 32, d, n, e, torch.full((d,), size, device="cuda"), new=new)
    o, _ = decode(fox, c, scale)
    for t in range(new):
        seen = n - (new - 1 - t)
        want = held(c) * (seen * 2.0**-e / (1 + seen * 2.0**-e))
        row = o[t::new].double()
        want = want[None, :, None].expand(64, -1, G, -1).reshape(row.shape)
        off = (row - want).abs() / want.abs()
        assert (off <= TOL).all(), (t, off.max().item())


@pytest.mark.parametrize("G,d", [(1, 128), (4, 64), (12, 64)])
@pytest.mark.parametrize("at", [3, 800])
def test_a_large_value_without_weight_in_the_same_channels(fox, G, d, at):
    """V of 30000 at a key that weighs nothing (2^-160): its scale is 2^19 times the others', whose weights of 2^-5 times that
    are 2^-24, within what 11 bits hold."""
    n, e = 1500, 5
    c, scale = sink(64, G, 32, d, n, e, torch.full((d,), 0.05, device="cuda"))
    for k, v, z in c.seq:
        k[at, :, 0], v[at] = -56.0, 30000.0  # 30000 * 2^-160 adds nothing
    o, _ = decode(fox, c, scale)
    check(o, c, n - 1, e)
