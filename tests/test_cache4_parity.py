"""The 4-bit cache on the GPU against its plain 64-bit form (fourtest.py).

Tolerances, fixed before the first run:
  K, V, scales and read-back values: the same bits (all of them follow from the inputs by one definition, with a
    single rounding each); slots that a call does not append to keep theirs.
  Q rotated: one rounding to bf16 (half a step, 2^-8 of the value) after fp32 products and a sum (three roundings of 2^-24 of
    |a| + |b| at most).
  g, gbase: as in the bf16 cache's tests (the same sums).
  O, LSE: the library's bounds for unit inputs, element by element (foxtest.o_check, TOL_*), against attention over the values
    that the cache holds.
"""
import pytest

import foxtest
from foxtest import assert_o, tensor_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FOX_ERR_DEVICE = 6


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    fox.lib()
    return fox


def Case4(*a, **kw):
    from fourtest import Case4

    return Case4(*a, **kw)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def angles(n, r, dev="cuda"):
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (
        -torch.arange(r // 2, dtype=torch.float64, device=dev) / (r // 2))
    return a.cos().float(), a.sin().float()


def near_rotated(got, src, cos, sin, pairs, at):
    from cachetest import rotate

    ref = rotate(src, cos[at : at + src.shape[0]], sin[at : at + src.shape[0]], pairs)
    top = src.double().abs().amax(-1, keepdim=True)
    return bool(((got.double() - ref).abs() <= 2**-8 * ref.abs() * (1 + 2**-20) + 6 * top * 2.0**-24).all())


def turner(cos, sin, pairs):
    from cachetest import rotate
    from fourtest import nearest_bf16

    def turn(k, at):
        r = 2 * cos.shape[1]
        y = rotate(k, cos[at : at + k.shape[0]], sin[at : at + k.shape[0]], pairs)
        return torch.cat([nearest_bf16(y[..., :r]), k[..., r:]], -1)

    return turn


# own, new, H, Hkv, d, page, more
APPENDS = [
    ([1], [1], 1, 1, 64, 16, dict()),                                                  # the first token
    ([17, None, 64, 5], [1, 1, 1, 1], 8, 2, 128, 16, dict(uniform=True, rot=128)),      # one idle, page edges
    ([16, 17, 33, 32], [1, 1, 2, 16], 4, 4, 64, 16, dict(rot=32, pairs=True, tail=3)),  # over a page's end
    ([40, 7, 200], [33, 0, 64], 6, 2, 128, 64, dict(rot=64)),                           # one brings nothing
    ([300, 129, None, 1000], [300, 129, 2, 871], 12, 4, 64, 32, dict(rot=64, pairs=True)),  # prompts, many pages
    ([1, 2, 3], [1, 2, 3], 40, 8, 128, 128, dict(rot=16)),                              # half a rotation within a block
    ([50, 128], [50, 1], 14, 2, 128, 64, dict(prefix=77, rot=128)),                     # behind a prefix, first own page
    ([31, 100], [31, 31], 4, 1, 64, 16, dict(prefix=32, uniform=True, rot=48)),         # partners across blocks
    ([2500], [2500], 2, 1, 64, 16, dict(rot=64)),                                       # 157 pages
    ([9, 30], [9, 2], 5, 1, 128, 32, dict(rot=96, pairs=True)),
    # Rows that threads take one after the other: two, four and eight, also where rows lie side by side in a block.
    ([700, 3], [600, 3], 32, 8, 128, 64, dict(rot=128)),
    ([1000, None, 301], [1000, 2, 301], 32, 8, 128, 16, dict(rot=64, pairs=True, tail=5)),
    ([2600, 17], [2600, 5], 16, 16, 128, 64, dict(rot=128)),
    ([9000, None, 1003], [9000, 1, 1003], 2, 1, 64, 128, dict(rot=64, pairs=True)),
]


@pytest.mark.parametrize("n", range(len(APPENDS)))
@pytest.mark.parametrize("strided,low", [(False, False), (True, True)])
def test_append(fox, n, strided, low):
    own, new, H, Hkv, d, S, more = APPENDS[n]
    more = dict(more)
    rot, pairs = more.pop("rot", 0), more.pop("pairs", False)
    c = Case4(own, new, H, Hkv, d, S, seed=n, low=low, **more)
    want = Case4(own, new, H, Hkv, d, S, seed=n, **more)
    cos, sin = angles(c.P + max([x or 0 for x in own]), rot) if rot else (None, None)
    turn = turner(cos, sin, pairs) if rot else None
    c.put(upto_new=False, turn=turn)
    want.put(turn=turn)
    k, v, z = c.new_rows()
    q, before = c.q, [x.clone() for x in (c.g, c.gbase)]
    if strided:  # rows of a joint projection's output
        joint = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k, v = (x.unflatten(1, (-1, d)) for x in joint.split([H * d, Hkv * d, Hkv * d], 1))
        z = torch.cat([z, z], 1)[:, H:]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kw = dict(cos=cos, sin=sin, pairs=pairs, ws=ws)
    if rot:
        kw.update(q=q, q_out=torch.full_like(c.q, float("nan")))
    for _ in range(2):  # the second call writes the same values again
        out = fox.fox_cache4_append(c.cache4(fox), c.batch(fox), k, v, z, **kw)
        assert fox.fox_check_error(ws) == 0
    for name in ("k4", "ks", "v4", "vs"):
        assert torch.equal(getattr(c, name), getattr(want, name)), name
    new_slot = torch.isnan(before[0]) & ~torch.isnan(want.g)  # [pages, H, S]
    assert torch.equal(bits(c.g)[~new_slot], bits(before[0])[~new_slot])
    fresh = torch.isnan(before[1]) & ~torch.isnan(want.gbase)
    assert torch.equal(bits(c.gbase)[~fresh], bits(before[1])[~fresh])
    tol = (8 + 11) * 2.0**-24
    got, ref = c.g.double()[new_slot], want.g.double()[new_slot]
    assert ((got - ref).abs() <= (tol + 2**-24) * ref.abs()).all()
    sel = fresh[..., 0]
    got, ref = c.gbase.double().sum(-1), want.gbase.double().sum(-1)
    assert ((got - ref).abs()[sel] <= (tol + 2**-23) * ref.abs()[sel]).all()
    for b in range(c.B):
        r = slice(c.row0[b], c.row0[b] + new[b])
        if rot and own[b] is None:
            assert torch.isnan(out[r]).all()
        elif rot:
            assert near_rotated(out[r], c.q[r], cos, sin, pairs, c.P + own[b] - new[b])
    if rot and c.rows > sum(new):
        assert torch.isnan(out[sum(new) :]).all()
    # What the cache holds, read back: the new rows, into strided outputs too, and every sequence whole.
    wide = torch.full((c.rows, 2, Hkv + 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    rk, rv = fox.fox_cache4_read(c.cache4(fox), c.batch(fox), k=wide[:, 0, 1:], v=wide[:, 1, 1:], ws=ws)
    assert fox.fox_check_error(ws) == 0 and torch.isnan(wide[:, :, 0]).all()
    for b in range(c.B):
        r = slice(c.row0[b], c.row0[b] + new[b])
        if own[b] is None:
            assert torch.isnan(rk[r]).all() and torch.isnan(rv[r]).all()
            continue
        for got, ref in ((rk, want.held[b][0]), (rv, want.held[b][1])):
            assert torch.equal(got[r].double(), ref[own[b] - new[b] :])
    assert torch.isnan(rk[sum(new) :]).all()
    have = [x or 0 for x in own]
    whole = fox.make_batch(c.lens, c.table, cu_new=torch.tensor([0] + have, device="cuda").cumsum(0).to(torch.int32),
                           max_new=max(have + [1]), prefix_table=c.ptable if c.P else None, prefix_len=c.P)
    rk, rv = fox.fox_cache4_read(c.cache4(fox), whole, sum(have), ws=ws)
    assert fox.fox_check_error(ws) == 0
    for i in range(2):
        ref = torch.cat([want.held[b][i] for b in range(c.B) if own[b] is not None])
        assert torch.equal((rk, rv)[i].double(), ref)


def hard_values(gen, n):
    """Rows of 32 bf16 values on every border: each scale's own seven steps, values halfway between codes and next to halfway,
    the largest and smallest that there are, zeros."""
    from fourtest import SCALES

    rows = []
    for s in SCALES[1:]:
        x = torch.tensor([7 * s] + [(u + 0.5) * s for u in range(7)] + [u * s for u in range(8)], dtype=torch.float64)
        near = torch.nextafter(x[1:8].bfloat16(), torch.tensor(0.0, dtype=torch.bfloat16)).double()
        rows.append(torch.cat([x, -x[1:8], near, torch.zeros(2, dtype=torch.float64)]))
        rows.append(torch.cat([torch.nextafter(x[:1].bfloat16(), torch.tensor(1e30, dtype=torch.bfloat16)).double().clamp(max=430080),
                               -x[1:16], near, -near, torch.zeros(2, dtype=torch.float64)]))
    rows.append(torch.zeros(32, dtype=torch.float64))
    rows.append(torch.full((32,), -430080.0, dtype=torch.float64))
    rows.append(torch.full((32,), 2.0**-120, dtype=torch.float64))
    rows.append(torch.cat([torch.tensor([2.0**-133]), torch.zeros(31)]).double())
    x = torch.stack(rows).bfloat16()
    random = (torch.randn(n, 32, generator=gen) * 2.0 ** torch.randint(-20, 16, (n, 1), generator=gen)).bfloat16()
    return torch.cat([x, random])


@pytest.mark.parametrize("d", [64, 128])
def test_every_border_of_the_form(fox, d):
    """All 248 scales, halves between codes, the ends of the range: bits and values as by the definition."""
    gen = torch.Generator().manual_seed(3)
    x = hard_values(gen, 3000)
    n = x.shape[0] // (d // 32) * (d // 32)
    x = x[:n].view(-1, 1, d)
    n = x.shape[0]
    c = Case4([n], [n], 1, 1, d, 64, seed=1)
    c.seq[0] = (x.cuda(), x.flip(0).cuda(), c.seq[0][2])
    want = Case4([n], [n], 1, 1, d, 64, seed=1)
    want.seq[0] = c.seq[0]
    want.put()
    k, v, z = c.new_rows()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fox.fox_cache4_append(c.cache4(fox), c.batch(fox), k, v, z, ws=ws)
    assert fox.fox_check_error(ws) == 0
    for name in ("k4", "ks", "v4", "vs"):
        assert torch.equal(getattr(c, name), getattr(want, name)), name
    rk, rv = fox.fox_cache4_read(c.cache4(fox), c.batch(fox), n, ws=ws)
    assert torch.equal(rk.double(), want.held[0][0]) and torch.equal(rv.double(), want.held[0][1])


def test_rotations_are_rounded_once(fox):
    """Angles and values for which a cos - b sin lies on, or 2^-24 of itself next to, a border between two bf16 values."""
    n, d = 4000, 128
    c = Case4([n], [n], 2, 2, d, 128, seed=2)
    g = torch.Generator().manual_seed(7)
    k = torch.randint(-255, 256, (n, 2, d), generator=g).float()
    k[::3] *= 2.0 ** -torch.randint(0, 12, k[::3].shape, generator=g)
    # cos with 8 bits and sin = 0, 1 or 2^-12: products that end on a half of bf16's step, or just beside it
    cos = torch.randint(1, 256, (n, d // 2), generator=g).float() / 256 + 2.0**-9
    sin = torch.tensor([0.0, 1.0, 2.0**-12, 2.0**-20])[torch.randint(0, 4, (n, d // 2), generator=g)]
    c.seq[0] = (k.bfloat16().cuda(), c.seq[0][1], c.seq[0][2])
    c.q = k.flip(0).bfloat16().cuda()
    cos, sin = cos.cuda(), sin.cuda()
    for pairs in (False, True):
        turn = turner(cos, sin, pairs)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        kn, vn, z = c.new_rows()
        out = fox.fox_cache4_append(c.cache4(fox), c.batch(fox), kn, vn, z, q=c.q, cos=cos, sin=sin, pairs=pairs, ws=ws)
        assert fox.fox_check_error(ws) == 0
        assert near_rotated(out, c.q, cos, sin, pairs, 0)
        want = Case4([n], [n], 2, 2, d, 128, seed=2)
        want.seq[0] = c.seq[0]
        want.put(turn=turn)
        assert torch.equal(c.k4, want.k4) and torch.equal(c.ks, want.ks)


def test_values_outside_the_form_are_reported(fox):
    """Infinities, NaN and magnitudes above 430080: reported, held as the nearest there is, the other blocks untouched."""
    for where in ("k", "v"):
        for bad, value in ((float("inf"), 430080.0), (-float("inf"), -430080.0), (float("nan"), 0.0), (1.0e6, 430080.0)):
            c = Case4([20], [20], 2, 2, 64, 16, seed=8)
            c.seq[0][0 if where == "k" else 1][7, 1, 40] = bad
            k, v, z = c.new_rows()
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            fox.fox_cache4_append(c.cache4(fox), c.batch(fox), k, v, z, ws=ws)
            assert fox.fox_check_error(ws) == FOX_ERR_DEVICE and fox.fox_check_error(ws) == 0
            got = dict(zip("kv", fox.fox_cache4_read(c.cache4(fox), c.batch(fox), 20, ws=ws)))
            assert all(torch.isfinite(x).all() for x in got.values())
            assert got[where][7, 1, 40].item() == value
            clean = Case4([20], [20], 2, 2, 64, 16, seed=8)
            clean.put()
            ref = torch.stack(clean.held[0])
            mine = torch.stack([got["k"], got["v"]]).double()
            same = torch.ones_like(ref, dtype=torch.bool)
            same["kv".index(where), 7, 1, 32:] = False
            assert torch.equal(mine[same], ref[same])


# own, new, H, Hkv, d, page, more
DECODES = [
    ([1], [1], 1, 1, 64, 16, dict()),                                             # one key
    ([1, 31, 32, 33], [1, 1, 1, 1], 4, 4, 128, 16, dict(uniform=True)),            # around a key tile
    ([None, 63, None, 64, 65], [1] * 5, 8, 2, 128, 64, dict(uniform=True)),        # idle ones between
    ([127, 128, 129, 500], [1] * 4, 8, 1, 64, 128, dict(uniform=True)),            # one key head
    ([9, 300, 77], [4, 2, 0], 14, 2, 128, 32, dict(tail=2)),                       # odd group, ragged new, rows behind
    ([13, 100], [13, 9], 6, 2, 64, 16, dict(bias_from_j=True)),                    # all keys are new
    ([70, 200], [5, 70], 8, 2, 128, 64, dict()),                                   # more rows than one row tile
    ([257, 1025], [3, 3], 16, 16, 64, 64, dict(uniform=True, bias_from_j=True)),
    ([1000, 3], [1, 1], 32, 8, 128, 64, dict(uniform=True, scale=0.3)),
    ([40, None, 1], [1, 1, 1], 8, 2, 128, 64, dict(uniform=True, prefix=300)),     # prefix of no whole pages
    ([33, 18], [2, 18], 6, 2, 64, 16, dict(prefix=64, tail=1)),
    ([5, 6, 7, 90], [1] * 4, 4, 4, 128, 32, dict(uniform=True, prefix=31, bias_from_j=True)),
    ([3] * 40, [1] * 40, 8, 2, 128, 16, dict(uniform=True, prefix=515)),           # many rows a key head
    ([20 + i % 3 for i in range(70)], [2] * 70, 12, 4, 64, 64, dict(prefix=200)),
    ([90, 700], [3, 1], 20, 1, 128, 64, dict()),                                   # a group wider than a row tile
    ([300, 44], [1, 1], 16, 2, 64, 128, dict(uniform=True, bias_from_j=True)),     # a full row tile
    ([70001], [1], 4, 1, 128, 64, dict()),                                         # long: split and joined
    ([30011, 5, 9000], [1, 3, 2], 8, 2, 64, 64, dict()),
    ([11], [1], 16, 16, 64, 64, dict(prefix=20000)),
    ([7, 130], [7, 6], 8, 2, 128, 64, dict(prefix=9999)),
    ([(b * 37) % 90 + 1 if b % 11 else None for b in range(600)], [1] * 600, 8, 4, 64, 16, dict(uniform=True)),
]


def check_decode(fox, c, label, bj=False, scale=None, want_prefix=None):
    cache, batch = c.cache4(fox), c.batch(fox)
    ws = fox.cache4_workspace(cache, batch, c.rows)
    ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF  # nothing is read that the call has not written
    o, lse = torch.full_like(c.q, float("nan")), torch.full((c.rows, c.H), float("nan"), device="cuda")
    fox.trace_begin()
    fox.fox_cache4_decode(cache, batch, c.q, scale=scale or 0.0, bias_from_j=bj, o=o, lse=lse, ws=ws)
    names = [k for k, _ in fox.trace_end()]
    assert want_prefix is None or ("prefix" in names) == want_prefix, names
    assert fox.fox_check_error(ws) == 0
    last = sum(c.new)
    assert torch.isnan(o[last:]).all() and torch.isnan(lse[last:]).all()
    ro, rl = c.attend(bias_from_j=bj, scale=scale)
    idle = torch.isinf(rl[:last])
    assert torch.equal(idle, torch.isinf(lse[:last])) and (o[:last][idle] == 0).all()
    if last:
        assert_o(tensor_f64(o[:last]), tensor_f64(ro[:last]), "bf16", label)
    if (~idle).any():
        assert (lse[:last].double() - rl[:last])[~idle].abs().max().item() <= foxtest.TOL_LSE_BF16
    # the same rows from a strided q, bit for bit
    H, d = c.H, c.d
    wide = torch.cat([c.q.flatten(1), c.q.flatten(1)], 1)[:, H * d :].unflatten(1, (H, d))
    o2, lse2 = fox.fox_cache4_decode(cache, batch, wide, scale=scale or 0.0, bias_from_j=bj, ws=ws)
    assert torch.equal(bits(o2[:last]), bits(o[:last])) and torch.equal(bits(lse2[:last]), bits(lse[:last]))
    return o, lse, ro, rl


@pytest.mark.parametrize("n", range(len(DECODES)))
def test_decode(fox, n):
    own, new, H, Hkv, d, S, more = DECODES[n]
    more = dict(more)
    bj, scale = more.pop("bias_from_j", False), more.pop("scale", None)
    c = Case4(own, new, H, Hkv, d, S, seed=50 + n, **more)
    c.put()
    check_decode(fox, c, f"decode4 {n}", bj, scale)


# Behind prefixes long enough for the batch that they are shared out (spread out, then one kernel for all sequences).
SHARED = [
    ([13 + i for i in range(48)], [1] * 48, 8, 8, 128, 64, 3001, dict(uniform=True, bias_from_j=True)),  # one row tile, keys split
    ([3] * 150, [1] * 150, 4, 1, 128, 16, 5003, dict(uniform=True)),                       # row tiles of a small group
    ([20 + i % 3 for i in range(170)], [2] * 170, 12, 4, 64, 64, 1537, dict(tail=3)),      # several, a tail of one key
    ([None if i % 5 == 2 else 6 + 11 * (i % 4) for i in range(164)], [1 + i % 5 for i in range(164)], 14, 2, 128, 32, 1664,
     dict(tail=1)),                                                                        # odd group, idle ones, no tail
    ([9] * 29, [1] * 29, 20, 1, 128, 128, 22001, dict(uniform=True, scale=0.2)),           # a group of two head chunks
    ([40, 5, 77, 300] * 4, [33, 5, 40, 1] * 4, 6, 2, 64, 16, 10002, dict(bias_from_j=True)),  # many new tokens
]


@pytest.mark.parametrize("n", range(len(SHARED)))
def test_decode_behind_a_shared_prefix(fox, n):
    own, new, H, Hkv, d, S, P, more = SHARED[n]
    more = dict(more)
    bj, scale = more.pop("bias_from_j", False), more.pop("scale", None)
    c = Case4(own, new, H, Hkv, d, S, seed=150 + n, prefix=P, **more)
    c.put()
    check_decode(fox, c, f"decode4 shared {n}", bj, scale, want_prefix=True)


def test_shared_values_outside_fp16_are_reported(fox):
    """The shared prefix's P V runs in fp16: a V held as 65536 or more there sets the error word; among a sequence's own tokens,
    or in a prefix that is walked, it is no error."""
    for B, P, status in ((150, 5003, FOX_ERR_DEVICE), (3, 100, 0)):
        for where in ("prefix", "own"):
            c = Case4([9] * B, [1] * B, 4, 1, 128, 16, uniform=True, prefix=P, seed=6)
            (c.pre if where == "prefix" else c.seq[1])[1][5, 0, 7] = 1.0e5
            c.put()
            cache, batch = c.cache4(fox), c.batch(fox)
            ws = fox.cache4_workspace(cache, batch, c.rows)
            fox.fox_cache4_decode(cache, batch, c.q, ws=ws)
            assert fox.fox_check_error(ws) == (status if where == "prefix" else 0)


@pytest.mark.parametrize("B,P", [(3, 100), (150, 5003)])
def test_bad_pages_of_a_prefix_are_reported(fox, B, P):
    """Page ids of the prefix outside the pool: reported, read as page 0 (finite here), nothing else."""
    c = Case4([9] * B, [1] * B, 4, 1, 128, 16, uniform=True, prefix=P, seed=6)
    for t in (c.k4, c.v4, c.ks, c.vs):
        t.zero_()
    c.put()
    for t in (c.g, c.gbase):
        t.nan_to_num_(0.0)
    c.ptable[1], c.ptable[2] = c.k4.shape[0], -1
    cache, batch = c.cache4(fox), c.batch(fox)
    ws = fox.cache4_workspace(cache, batch, c.rows)
    fox.fox_cache4_decode(cache, batch, c.q, ws=ws)
    assert fox.fox_check_error(ws) == FOX_ERR_DEVICE
    assert fox.fox_check_error(ws) == 0


@pytest.mark.parametrize("H,d,S", [(16, 64, 16), (9, 128, 32), (8, 128, 64), (1, 64, 128)])
def test_decode_of_the_most_sequences(fox, H, d, S):
    """2048 of them: the most shared memory that a call takes."""
    own = [b % 35 + 1 if b % 7 else None for b in range(2048)]
    c = Case4(own, [1] * 2048, H, 1, d, S, uniform=True, seed=10)
    c.put()
    check_decode(fox, c, "decode4 most")


@pytest.mark.parametrize("gain_k,gain_v", [(1.0, 2.0**-16), (1.0, 3000.0), (6.0, 1.0), (2.0**-10, 2.0**-10), (40.0, 1.0)])
def test_scales_of_every_size(fox, gain_k, gain_v):
    """V a few steps above the least scale, or near the largest of fp16's values; scores that peak. O rounded by half a step,
    2^-8 of itself at most; a weight and its product with a scale by 2^-11 each, so 2^-10 of the largest V over all of them; and scores of
    40 sigma in fp32: a block's sum stands some 1060 |q| high (16 channels times 264, 16 times 24, random signs), 2^-23 of which times
    s / sqrt(d) = 16 / 11.3 is 1.8e-4, of four blocks 3.6e-4; a weight off by that moves O by twice it at most: 2^-10 of the largest V."""
    c = Case4([900, 33], [1, 2], 8, 2, 128, 64, seed=31)
    for b in range(2):
        k, v, z = c.seq[b]
        c.seq[b] = ((k * gain_k).bfloat16(), (v * gain_v).bfloat16(), z)
    c.put()
    cache, batch = c.cache4(fox), c.batch(fox)
    o, lse = fox.fox_cache4_decode(cache, batch, c.q)
    ro, rl = c.attend()
    most = torch.cat([c.held[b][1].abs().amax().view(1) for b in range(2)]).amax()
    assert ((o.double() - ro).abs() <= 2.0**-8 * ro.abs() + 2.0**-9 * most).all()
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16 * max(1.0, gain_k / 4)


@pytest.mark.parametrize("d", [64, 128])
def test_scales_that_differ_by_block_and_rise_along_the_sequence(fox, d):
    """V's blocks of very different sizes, the largest token last (the running reference moves) or first: each block of O to its
    own size, where its values are not below 2^-20 of the largest scale of the tile times the weight. O rounded by 2^-8 of itself; weights and
    products by 2^-11 each, of a weighted mean of |V| / block, which sizes of 1/4 to 4 keep below 4: 2^-10 of that, and as much for scores."""
    for back in (False, True):
        n = 500
        c = Case4([n], [1], 4, 2, d, 32, seed=32)
        k, v, z = c.seq[0]
        size = torch.logspace(-2, 2, n, base=2.0, device="cuda")
        size = size.flip(0) if back else size
        block = 2.0 ** (-3.0 * torch.arange(d // 32, device="cuda")).repeat_interleave(32)
        c.seq[0] = (k, (v * size[:, None, None] * block).bfloat16(), z + 6)
        c.put()
        o, lse = fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), c.q)
        ro, rl = c.attend()
        err = (o.double() - ro).abs() / block
        assert (err <= 2.0**-8 * (ro.abs() / block) + 2.0**-9 * 4).all()
        assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


def test_scores_that_rise_along_the_sequence(fox):
    """The running maximum is passed over and over."""
    n = 3000
    c = Case4([n, 70], [1, 1], 8, 2, 128, 64, seed=33, uniform=True, z_mean=9.0)
    k, v, z = c.seq[0]
    grow = 1 + 12 * torch.arange(n, device="cuda") / n
    c.seq[0] = ((k.float() * grow[:, None, None]).bfloat16(), v, z + 9)
    c.put()
    o, lse = fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 rising")
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


def test_queries_of_every_size(fox):
    """q from 2^-100 to 2^60 against a scale that undoes it: scores as of unit queries, in fp32."""
    for e in (-100, -30, 0, 15, 60):
        c = Case4([200, 3], [1, 2], 8, 2, 64, 16, seed=34)
        c.put()
        c.q = (c.q * 2.0**e).bfloat16()
        scale = 2.0**-e / 8
        o, lse = fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), c.q, scale=scale)
        ro, rl = c.attend(scale=scale)
        assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 q sizes")
        assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


def test_many_small_weights_count(fox):
    """One key of weight 1 and 100000 of 2^-24 whose values agree: O is 0.6 by these alone. Weights in fp16 at 2^11 times their
    value hold 2^-24 with 11 bits (2^-11), scales take one more rounding (2^-11), and O is rounded by 2^-8 of itself: 2^-8 + 2^-10 of O."""
    n, d = 100000, 64
    c = Case4([n], [1], 1, 1, d, 128, uniform=True, seed=5)
    k, v, z = c.seq[0]
    k.zero_()
    k[n // 3] = 2.1  # held as 2.0 or more: the weight below follows from what is held
    v.fill_(112.0)
    v[n // 3] = 0.0
    z.fill_(float("inf"))
    c.q.fill_(1.0)
    c.put()
    o, lse = fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert 0.2 < ro.min().item() and ro.max().item() < 2.0
    assert ((o.double() - ro).abs() <= (2.0**-8 + 2.0**-10) * ro.abs() + 1e-4).all()
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


def test_appending_and_decoding_a_sequence(fox):
    """Prompts in one call, then steps of one and several tokens, each appended with rotated keys and attended to at once:
    as one plain computation over everything that was appended."""
    H, Hkv, d, S, rot = 8, 2, 128, 32, 64
    prompt, steps = [70, 33], [1, 1, 3, 1, 2, 1]
    total = [x + sum(steps) for x in prompt]
    cos, sin = angles(max(total), rot)
    turn = turner(cos, sin, False)
    c = Case4(total, [1, 1], H, Hkv, d, S, seed=40, low=True)
    want = Case4(total, [1, 1], H, Hkv, d, S, seed=40)
    want.put(turn=turn)
    cache = c.cache4(fox)
    at = [0, 0]
    for n in [prompt] + [[s, s] for s in steps]:
        rows = [torch.cat([c.seq[b][i][at[b] : at[b] + n[b]] for b in range(2)]) for i in range(3)]
        at = [x + y for x, y in zip(at, n)]
        lens = torch.tensor(at, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda")
        batch = fox.make_batch(lens, c.table, cu_new=cu, max_new=max(n))
        q = torch.randn(sum(n), H, d, device="cuda", generator=c.gen).bfloat16()
        ws = fox.cache4_workspace(cache, batch, sum(n))
        turned = fox.fox_cache4_append(cache, batch, *rows, q=q, cos=cos, sin=sin, ws=ws)
        o, lse = fox.fox_cache4_decode(cache, batch, turned, ws=ws)
        assert fox.fox_check_error(ws) == 0
        ref = Case4(at, n, H, Hkv, d, S, seed=1)
        ref.seq = [tuple(x[: at[b]] for x in c.seq[b]) for b in range(2)]
        ref.held = {-1: (ref.pre[0], ref.pre[1]), **{b: tuple(x[: at[b]] for x in want.held[b]) for b in range(2)}}
        ref.q = turned
        ro, rl = ref.attend()
        assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 steps")
        assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16
    assert torch.equal(c.k4, want.k4) and torch.equal(c.v4, want.v4)


def test_stale_slots_and_later_tokens_do_not_count(fox):
    """Several new tokens: no row sees what lies behind it. Slots behind the ends hold all ones (NaN scales) by the helper."""
    own, new = [77, 40], [5, 40]
    a = Case4(own, new, 8, 2, 64, 16, seed=60)
    a.put()
    o, lse = fox.fox_cache4_decode(a.cache4(fox), a.batch(fox), a.q)
    b = Case4(own, new, 8, 2, 64, 16, seed=60)
    for i in range(2):
        k, v, z = b.seq[i]
        k[-1] *= 3
        v[-1] *= 1000
        z[-1] = -50.0
    b.put()
    o2, lse2 = fox.fox_cache4_decode(b.cache4(fox), b.batch(fox), b.q)
    last = [sum(new[: i + 1]) - 1 for i in range(2)]
    keep = [i for i in range(a.rows) if i not in last]
    ro, rl = a.attend()
    assert_o(tensor_f64(o2[keep]), tensor_f64(ro[keep]), "bf16", "decode4 later tokens")
    assert (lse2[keep].double() - rl[keep]).abs().max().item() <= foxtest.TOL_LSE_BF16


@pytest.mark.parametrize("prefix", [0, 40])
def test_pages_beyond_32_bit_offsets(fox, prefix):
    """A pool of 2^32 bytes and more, the pages in use at its end."""
    pages = (1 << 32) // (8 * 128 * 64) + 40
    c = Case4([300, 17], [2, 17], 16, 8, 128, 128, pages=pages, prefix=prefix, seed=4)
    c.put(upto_new=False)
    held = dict(c.held)
    k, v, z = c.new_rows()
    cache, batch = c.cache4(fox), c.batch(fox)
    ws = fox.cache4_workspace(cache, batch, c.rows)
    fox.fox_cache4_append(cache, batch, k, v, z, ws=ws)
    o, lse = fox.fox_cache4_decode(cache, batch, c.q, ws=ws)
    rk, rv = fox.fox_cache4_read(cache, batch, c.rows, ws=ws)
    assert fox.fox_check_error(ws) == 0
    want = Case4([300, 17], [2, 17], 16, 8, 128, 128, seed=4, prefix=prefix)
    want.pre, want.seq = c.pre, c.seq
    want.put()
    assert torch.equal(rk.double(), torch.cat([want.held[0][0][-2:], want.held[1][0]]))
    c.held = want.held
    assert torch.equal(held[0][0], want.held[0][0][:-2])
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 far pages")
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


@pytest.mark.parametrize("prefix", [0, 100])
def test_what_the_batch_cannot_hold_is_reported_and_skipped(fox, prefix):
    own, new = [40, 70, 33], [2, 2, 2]

    def fresh():
        c = Case4(own, new, 4, 2, 64, 16, seed=21, prefix=prefix)
        for t in (c.k4, c.v4, c.ks, c.vs):
            t.zero_()
        c.put(upto_new=False)
        c.g.nan_to_num_(0.0)
        c.gbase.nan_to_num_(0.0)
        return c

    good = fresh()
    k, v, z = good.new_rows()
    fox.fox_cache4_append(good.cache4(fox), good.batch(fox), k, v, z)
    for what in ("page", "negative page", "too long", "negative length", "in the prefix", "falling rows"):
        c = fresh()
        if what == "page":
            c.table[1, 4] = c.k.shape[0]
        elif what == "negative page":
            c.table[1, 4] = -2
        elif what == "too long":
            c.lens[1] = prefix + c.width * 16 + 1
        elif what == "negative length":
            c.lens[1] = -5
        elif what == "in the prefix":
            c.lens[1] = prefix + 1
        else:
            c.cu[2] = 1
        cache, batch = c.cache4(fox), c.batch(fox)
        ws = fox.cache4_workspace(cache, batch, c.rows)
        fox.fox_cache4_append(cache, batch, k, v, z, ws=ws)
        assert fox.fox_check_error(ws) == FOX_ERR_DEVICE, what
        o, lse = fox.fox_cache4_decode(cache, batch, c.q, ws=ws)
        assert fox.fox_check_error(ws) == FOX_ERR_DEVICE, what
        rk, rv = fox.fox_cache4_read(cache, batch, c.rows, ws=ws)
        assert fox.fox_check_error(ws) == FOX_ERR_DEVICE, what
        assert fox.fox_check_error(ws) == 0
        rows = [0, 1] if what == "falling rows" else [0, 1, 4, 5]
        full = Case4(own, new, 4, 2, 64, 16, seed=21, prefix=prefix)
        full.put()
        ro, rl = full.attend()
        assert_o(tensor_f64(o[rows]), tensor_f64(ro[rows]), "bf16", f"decode4 beside {what}")
        assert (lse[rows].double() - rl[rows]).abs().max() <= foxtest.TOL_LSE_BF16, what
        assert torch.equal(rk[:2].double(), full.held[0][0][-2:]), what
        ids = torch.cat([good.table[0, :3], good.table[2, :3]]) if what != "falling rows" else good.table[0, :3]
        for x, y in ((c.k4, good.k4), (c.v4, good.v4), (c.ks, good.ks), (c.vs, good.vs), (c.g, good.g)):
            assert torch.equal(bits(x[ids.long()]), bits(y[ids.long()])), what


def test_captured_steps_are_replayed_on_new_contents(fox):
    """An append and a decode in a graph; between replays lengths, rows and tables change."""
    H, Hkv, d, S, B = 8, 2, 128, 32, 3
    c = Case4([100, 64, 9], [1] * B, H, Hkv, d, S, uniform=True, seed=70)
    c.put(upto_new=False)
    cache, batch = c.cache4(fox), c.batch(fox)
    ws = fox.cache4_workspace(cache, batch, B)
    k, v, z = c.new_rows()
    o, lse = torch.empty_like(c.q), torch.empty(B, H, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            fox.fox_cache4_append(cache, batch, k, v, z, ws=ws, stream=side)
            fox.fox_cache4_decode(cache, batch, c.q, o=o, lse=lse, ws=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for idle in (None, 1):
        d2 = Case4([100, 64 if idle is None else None, 9], [1] * B, H, Hkv, d, S, uniform=True, seed=70)
        if idle is not None:
            c.lens[idle] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert fox.fox_check_error(ws) == 0
        d2.seq, d2.q = c.seq, c.q
        full = Case4([100, 64, 9], [1] * B, H, Hkv, d, S, uniform=True, seed=70)
        full.put()
        d2.held = full.held
        ro, rl = d2.attend()
        assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 graph")
        live = ~torch.isinf(rl)
        assert (lse.double() - rl)[live].abs().max().item() <= foxtest.TOL_LSE_BF16 and torch.equal(live, ~torch.isinf(lse))


def test_two_batches_at_once_on_their_own_streams_and_workspaces(fox):
    cases = [Case4([400 + 100 * i, 77], [1, 2], 8, 2, 64, 16, seed=80 + i) for i in range(2)]
    for c in cases:
        c.put()
    ws = [fox.cache4_workspace(c.cache4(fox), c.batch(fox), c.rows) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    out = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate(cases):
            out[i].append(fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), c.q, ws=ws[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        assert fox.fox_check_error(ws[i]) == 0
        ro, rl = c.attend()
        for o, lse in out[i]:
            assert torch.equal(bits(o), bits(out[i][0][0])) and torch.equal(bits(lse), bits(out[i][0][1]))
        assert_o(tensor_f64(out[i][0][0]), tensor_f64(ro), "bf16", "decode4 streams")


def test_a_captured_decode_behind_a_shared_prefix_is_replayed(fox):
    """The prefix is spread out in the workspace by the graph itself: what another call left there, and other tokens in the pool,
    make no difference to a replay but the tokens' own."""
    B, P = 150, 5003
    c = Case4([3] * B, [1] * B, 4, 1, 128, 16, uniform=True, seed=90, prefix=P)
    c.put()
    cache, batch = c.cache4(fox), c.batch(fox)
    ws = fox.cache4_workspace(cache, batch, B)
    o, lse = torch.empty_like(c.q), torch.empty(B, 4, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        fox.fox_cache4_decode(cache, batch, c.q, o=o, lse=lse, ws=ws, stream=side)
    for i in range(2):
        if i:  # other tokens in the same pages
            other = Case4([3] * B, [1] * B, 4, 1, 128, 16, uniform=True, seed=91, prefix=P)
            c.pre, c.seq = other.pre, other.seq
            c.put()
            ws[fox.FOX_CACHE_ZERO_BYTES:].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert fox.fox_check_error(ws) == 0
        direct, dl = fox.fox_cache4_decode(cache, batch, c.q)
        assert torch.equal(bits(o), bits(direct)) and torch.equal(bits(lse), bits(dl))
        ro, rl = c.attend()
        assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 shared graph")
        assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


def test_threads_of_the_host_call_at_once(fox):
    """Appends, decodes and reads of four threads, each with its own cache, stream and workspace."""
    import threading

    cases = [Case4([200 + 30 * i, 50], [2, 1], 8, 2, 128, 32, seed=100 + i) for i in range(4)]
    for c in cases:
        c.put()
    torch.cuda.synchronize()
    results, errors = [None] * 4, []

    def work(i):
        try:
            c, s = cases[i], torch.cuda.Stream()
            cache, batch = c.cache4(fox), c.batch(fox)
            with torch.cuda.stream(s):
                ws = fox.cache4_workspace(cache, batch, c.rows)
                k, v, z = c.new_rows()
                for _ in range(30):
                    fox.fox_cache4_append(cache, batch, k, v, z, ws=ws, stream=s)
                    out = fox.fox_cache4_decode(cache, batch, c.q, ws=ws, stream=s)
                    read = fox.fox_cache4_read(cache, batch, c.rows, ws=ws, stream=s)
            s.synchronize()
            results[i] = (out, read, fox.fox_check_error(ws, s))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for c, ((o, lse), (rk, rv), status) in zip(cases, results):
        assert status == 0
        ro, rl = c.attend()
        assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode4 threads")
        for b in range(c.B):
            r, n = slice(c.row0[b], c.row0[b] + c.new[b]), c.own[b] - c.new[b]
            assert torch.equal(rk[r].double(), c.held[b][0][n:]) and torch.equal(rv[r].double(), c.held[b][1][n:])


def test_without_the_extension(fox, monkeypatch):
    """The same calls by way of ctypes."""
    c = Case4([40, 20], [1, 3], 4, 2, 64, 16, seed=3, low=True)
    c.put()
    cache, batch = c.cache4(fox), c.batch(fox)
    cos, sin = angles(64, 32)

    def calls():
        k, v, z = c.new_rows()
        q = fox.fox_cache4_append(cache, batch, k, v, z, q=c.q, cos=cos, sin=sin)
        fox.fox_cache4_append(cache, batch, k, v, z)
        return [q, *fox.fox_cache4_decode(cache, batch, c.q, scale=0.3), *fox.fox_cache4_read(cache, batch, c.rows)]

    first = calls()
    monkeypatch.setattr(fox, "_call", fox._CtypesCall)
    for x, y in zip(first, calls()):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("H,Hkv,d,new,bad", [(8, 2, 128, 1, float("nan")), (32, 2, 64, 1, float("inf")), (4, 1, 128, 3, float("-inf"))])
def test_a_bad_query_row_stays_alone(fox, H, Hkv, d, new, bad):
    """A NaN or an infinity in one row of q: the rows that share its tiles are as without it."""
    c = Case4([900, 40], [new] * 2, H, Hkv, d, 32, seed=130, uniform=True)
    c.put()
    ro, rl = c.attend()
    q = c.q.clone()
    q[0, 1, 5] = bad
    o, lse = fox.fox_cache4_decode(c.cache4(fox), c.batch(fox), q)
    sound = torch.ones(c.rows, H, dtype=torch.bool, device="cuda")
    sound[0, 1] = False
    assert_o(tensor_f64(o[sound]), tensor_f64(ro[sound]), "bf16", "decode4 beside a bad row")
    assert (lse.double() - rl)[sound].abs().max().item() <= foxtest.TOL_LSE_BF16
    assert not torch.isfinite(lse[0, 1]) or not torch.isfinite(o[0, 1]).all()


def test_handles_of_the_other_kind_are_refused(fox):
    """The calls read the handle's C struct, and the two kinds' differ."""
    c = Case4([40, 20], [1, 1], 4, 2, 64, 16, uniform=True, seed=3)
    four, batch, rows = c.cache4(fox), c.batch(fox), c.new_rows()
    bf16 = fox.make_cache(c.k, c.v, c.g, c.gbase)
    for call, cache in ((fox.fox_cache4_append, bf16), (fox.fox_cache_append, four)):
        with pytest.raises(TypeError):
            call(cache, batch, *rows)
    for call, cache in ((fox.fox_cache4_decode, bf16), (fox.fox_decode, four)):
        with pytest.raises(TypeError):
            call(cache, batch, c.q)
    with pytest.raises(TypeError):
        fox.fox_cache4_read(bf16, batch, 2)


def test_binding_refusals(fox):
    c = Case4([40, 20], [1, 1], 4, 2, 64, 16, uniform=True, seed=3)
    cache, batch = c.cache4(fox), c.batch(fox)
    k, v, z = c.new_rows()
    with pytest.raises(TypeError):
        fox.fox_cache4_decode(cache, batch, c.q.float())
    with pytest.raises(ValueError):
        fox.fox_cache4_decode(cache, batch, c.q[:, :2])
    with pytest.raises(fox.FoxError):
        fox.fox_cache4_decode(cache, batch, c.q, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fox.FoxError):
        fox.fox_cache4_decode(cache, batch, c.q, o=c.q)
    with pytest.raises(ValueError):
        fox.fox_cache4_append(cache, batch, k, v, z[:, :3])
    with pytest.raises(TypeError):
        fox.fox_cache4_append(cache, batch, k.float(), v, z)
    with pytest.raises(ValueError):
        fox.fox_cache4_read(cache, batch)
    with pytest.raises(fox.FoxError):
        fox.fox_cache4_read(cache, batch, k=k, v=k)
    with pytest.raises(TypeError):
        fox.fox_cache4_read(cache, batch, k=k.float())
    with pytest.raises(ValueError):
        fox.make_cache4(c.k4, c.v4[:1], c.ks, c.vs, c.g, c.gbase)
    with pytest.raises(ValueError):
        fox.make_cache4(c.k4, c.v4, c.ks, c.vs[:, :, :, :2], c.g, c.gbase)
    with pytest.raises(TypeError):
        fox.make_cache4(c.k4.int(), c.v4, c.ks, c.vs, c.g, c.gbase)
    made = fox.new_cache4(4, 16, 8, 2, 128)
    assert made.g_low is not None and made.d == 128
