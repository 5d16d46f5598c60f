"""LSE of the decode over the 4-bit cache, to what fp32 sums of the scores allow.

A block's score is a sum of n q (n = u + 8, 1 .. 15) over its 32 channels, less 8 times the sum of q, times the scale s: two matrix products of
16 channels, one of the sums of q with the scales, and sums over the blocks in fp32. A matrix product aligns its 16 terms and what it is
added to by the exponents of the largest: 256 |q| (codes at bits 5..2 of an operand without exponent stand 256 units high) or the sum so far;
each is cut off at 2^-25 of it, the sum at 2^-23 of itself. So with M = max(256 max |q|, sum n |q|) a product is off by 17 * 2^-25 M + 2^-23 M =
21 * 2^-25 M, a block by twice that, the product of the scales by no more than one of them, and NB + 1 additions by 2^-24 M each:
48 * 2^-25 M s a block and as much for the rest cover all of it. An exponential adds 2^-22, LSE's own sum and logarithm 2^-22 of LSE, and gates,
which are open here (|g| below 1), 2^-23."""
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


def heights(c, scale, floor):
    """The largest sum of M s of a row over the keys, with max |q| times `floor` in M: [rows, H]."""
    from fourtest import SCALES

    out = torch.zeros(c.rows, c.H, dtype=torch.float64, device="cuda")
    table = torch.tensor(SCALES, dtype=torch.float64, device="cuda")
    G = c.H // c.Hkv
    for b in range(c.B):
        x = torch.cat([c.held[-1][0], c.held[b][0]]).unflatten(-1, (-1, 32))  # [keys, Hkv, blocks, 32]
        s = table[torch.searchsorted(7 * table, x.abs().amax(-1).contiguous())]
        n = x / torch.where(s > 0, s, 1.0)[..., None] + 8
        r = slice(c.row0[b], c.row0[b] + c.new[b])
        q = c.q[r].double().abs().view(-1, c.Hkv, G, c.d // 32, 32)
        sums = torch.einsum("rhgbc,jhbc->jrhgb", q, n)
        m = torch.maximum(sums, floor * q.amax(-1))
        out[r] = (m * s[:, None, :, None]).sum(-1).amax(0).flatten(1)
    return out * scale


def lse_and_reference(fox, c, scale):
    c.put()
    o, lse = fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), c.q, scale=scale)
    ro, rl = c.attend(scale=scale)
    return lse.double(), rl, 2.0**-22 + 2.0**-23 + 2.0**-22 * rl.abs().clamp(min=1.0)


SHAPES = [(1, 128, 64), (4, 128, 64), (4, 64, 16), (8, 64, 32), (8, 128, 128), (14, 128, 64), (12, 64, 16)]


@pytest.mark.parametrize("G,d,S", SHAPES)
@pytest.mark.parametrize("q_of", ["one sign", "normal", "few large"])
@pytest.mark.parametrize("size", [1.0, 2.0**-9, 300.0])
def test_lse(fox, G, d, S, q_of, size):
    from fourtest import Case4

    c = Case4([1000, 33, 1], [1, 2, 1], 2 * G, 2, d, S, seed=11)
    c.seq = [((k * size).bfloat16(), v, z + 9) for k, v, z in c.seq]
    if q_of == "one sign":  # sums of q as large as they come
        c.q = c.q.abs()
        c.q[:, ::2] *= -1
    elif q_of == "few large":
        c.q[..., 5::32] *= 40
    scale = d**-0.5 / size / (8 if q_of == "few large" else 1)
    lse, rl, tol = lse_and_reference(fox, c, scale)
    off = (lse - rl).abs() / (2 * 48 * 2.0**-25 * heights(c, scale, 256) + tol)
    assert (off <= 1).all(), off.max().item()


@pytest.mark.parametrize("G,d,S", SHAPES)
def test_lse_of_queries_whose_block_sums_are_exact(fox, G, d, S):
    """Of q every other channel is a multiple of 2^-5 in [4, 8), the others odd multiples of 2^-13 below 2^-5, all of one sign. Terms are multiples of
    2^-13, which no term of 2^11 (256 * 8) or sum of 2^11 (32 channels of 15 and 8, half of them) cuts off, and the sums of q, 8 * 2^-13 of them at
    most 2^10, are exact in two fp16. What is left are the sums of blocks in fp32: NB + 1 additions, 2^-24 of sum n |q| s each."""
    from fourtest import Case4

    c = Case4([1000, 33, 1], [1, 2, 1], 2 * G, 2, d, S, seed=12)
    c.seq = [(k, v, z + 9) for k, v, z in c.seq]
    large = torch.randint(128, 256, c.q.shape, generator=c.gen, device="cuda") / 32
    small = (torch.randint(0, 128, c.q.shape, generator=c.gen, device="cuda") * 2 + 1) / 8192
    q = torch.where(torch.arange(d, device="cuda") % 2 == 1, large, small)
    q[:, ::2] *= -1
    c.q = q.bfloat16()
    assert torch.equal(c.q.double(), q.double())
    scale = d**-0.5 / 8
    lse, rl, tol = lse_and_reference(fox, c, scale)
    off = (lse - rl).abs() / ((d // 32 + 1) * 2.0**-24 * heights(c, scale, 0) + tol)
    assert (off <= 1).all(), off.max().item()
