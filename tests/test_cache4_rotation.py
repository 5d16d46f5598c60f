"""K's rotation where the two products differ so much that 64 bits do not hold their difference: a cos on a border between two bf16 values, b sin
2^-50 to 2^-110 of it, on either side. By fractions of whole numbers, to the nearest bf16; codes and scales bit for bit."""
from fractions import Fraction

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    fox.lib()
    return fox


def nearest(x):
    """A fraction to the nearest number of 8 significant bits, ties to even."""
    if x == 0:
        return 0.0
    e = 0
    while abs(x) >= Fraction(2) ** (e + 1):
        e += 1
    while abs(x) < Fraction(2) ** e:
        e -= 1
    step = Fraction(2) ** (e - 7)
    return float(round(x / step) * step)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_products_far_apart(fox, d, pairs):
    from fourtest import Case4

    n, half = 60, d // 2
    gen = torch.Generator().manual_seed(4)
    # 149 / 256 * 3 / 4 = 447 / 1024: halfway between the bf16 values 7 / 16, where a code of scale 1 / 8 begins, and the one below
    a = torch.full((n, half), 149 / 256) * (torch.randint(0, 2, (n, half), generator=gen) * 2 - 1)
    cos = torch.full((n, half), 0.75)
    sin = 0.5 + torch.rand(n, half, generator=gen) / 4
    b = (1 + torch.rand(n, half, generator=gen)) * 2.0 ** -torch.randint(50, 110, (n, half), generator=gen)
    b *= torch.randint(0, 2, (n, half), generator=gen) * 2 - 1
    # every fourth pair is not turned: 7 / 8, which sets the block's scale
    a[:, ::4], b[:, ::4], cos[:, ::4], sin[:, ::4] = 0.875, 0.875, 1.0, 0.0
    a, b = a.bfloat16(), b.bfloat16()
    k = torch.stack([a, b], -1).flatten(1) if pairs else torch.cat([a, b], 1)
    u, w = torch.empty(n, half), torch.empty(n, half)
    for t in range(n):
        for i in range(half):
            x, y, c, s = (Fraction(float(z[t, i])) for z in (a, b, cos, sin))
            u[t, i], w[t, i] = nearest(x * c - y * s), nearest(y * c + x * s)
    turned = (torch.stack([u, w], -1).flatten(1) if pairs else torch.cat([u, w], 1)).cuda()[:, None].bfloat16()
    # the rounding in question goes both ways
    at_border = turned.float().abs().flatten()
    assert (at_border == 7 / 16).any() and (at_border == 7 / 16 - 2.0**-9).any()
    c = Case4([n], [n], 1, 1, d, 64, seed=1)
    c.seq[0] = (k.cuda()[:, None], c.seq[0][1], c.seq[0][2])
    want = Case4([n], [n], 1, 1, d, 64, seed=1)
    want.seq[0] = c.seq[0]
    want.put(turn=lambda k, at: turned[: k.shape[0]])
    kn, vn, z = c.new_rows()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fox.fox_cache4_append(c.cache4(fox), c.batch(fox), kn, vn, z, cos=cos.cuda(), sin=sin.cuda(), pairs=pairs, ws=ws)
    assert fox.fox_check_error(ws) == 0
    assert torch.equal(c.ks, want.ks) and torch.equal(c.k4, want.k4)
