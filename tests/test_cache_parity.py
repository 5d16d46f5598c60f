"""The paged cache on the GPU against its plain 64-bit form (cachetest.py).

Tolerances, fixed before the first run:
  V, and every slot that the call does not append to: the same bits (stale slots hold NaN).
  K and Q rotated: one rounding to the cache's type (half a step, eps / 2 of the value) after fp32
    products and a sum (three roundings of 2^-24 of |a| + |b| at most).
  g: fp32 sums of terms of one sign: log sigmoid within 8 * 2^-24 of itself (two library functions
    of at most 2 ulp, an addition), a scan of at most 4 + 5 + 2 additions, plus one addition an earlier call.
  gbase: sums of such g, in fp64.
  O, LSE: the library's bounds for unit inputs, element by element (foxtest.o_check, TOL_*).
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


def Case(*a, **kw):
    from cachetest import Case

    return Case(*a, **kw)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def angles(n, r, dev="cuda"):
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (
        -torch.arange(r // 2, dtype=torch.float64, device=dev) / (r // 2))
    return a.cos().float(), a.sin().float()


# own, new, H, Hkv, d, page, more
APPENDS = [
    ([1], [1], 1, 1, 64, 16, dict()),                                                  # the first token
    ([17, None, 64, 5], [1, 1, 1, 1], 8, 2, 128, 16, dict(uniform=True, rot=128)),      # one idle, page edges
    ([16, 17, 33, 32], [1, 1, 2, 16], 4, 4, 64, 16, dict(rot=32, pairs=True, tail=3)),  # over a page's end
    ([40, 7, 200], [33, 0, 64], 6, 2, 128, 64, dict(rot=64)),                           # one brings nothing
    ([300, 129, None, 1000], [300, 129, 2, 871], 12, 4, 64, 32, dict(rot=64, pairs=True)),  # prompts, many pages
    ([1, 2, 3], [1, 2, 3], 40, 8, 128, 128, dict(rot=16)),                              # more heads than one gate block
    ([50, 128], [50, 1], 14, 2, 128, 64, dict(prefix=77, rot=128)),                     # behind a prefix, first own page
    ([31, 100], [31, 31], 4, 1, 64, 16, dict(prefix=32, uniform=True)),                 # prefix ends with its page
    ([2500], [2500], 2, 1, 64, 16, dict()),                                             # 157 pages: five scan steps
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", range(len(APPENDS)))
@pytest.mark.parametrize("strided", [False, True])
def test_append(fox, n, dtype, strided):
    own, new, H, Hkv, d, S, more = APPENDS[n]
    more = dict(more)
    rot, pairs = more.pop("rot", 0), more.pop("pairs", False)
    c = Case(own, new, H, Hkv, d, S, dtype=dtype, seed=n, **more)
    c.put(upto_new=False)
    k, v, z = c.new_rows()
    q, before = c.q, [x.clone() for x in (c.k, c.v, c.g, c.gbase)]
    want = Case(own, new, H, Hkv, d, S, dtype=dtype, seed=n, **more)
    want.put()
    if strided:  # rows of a joint projection's output
        joint = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k, v = (x.unflatten(1, (-1, d)) for x in joint.split([H * d, Hkv * d, Hkv * d], 1))
        z = torch.cat([z, z], 1)[:, H:]
    cos, sin = angles(c.P + max([x or 0 for x in own]), rot) if rot else (None, None)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kw = dict(cos=cos, sin=sin, pairs=pairs, ws=ws)
    if rot:
        kw.update(q=q, q_out=torch.full_like(c.q, float("nan")))
    for _ in range(2):  # the second call writes the same values again
        out = fox.fox_cache_append(c.cache(fox), c.batch(fox), k, v, z, **kw)
        assert fox.fox_check_error(ws) == 0
    assert torch.equal(bits(c.v), bits(want.v))
    # slots that the call appends to
    new_slot = torch.isnan(before[2]) & ~torch.isnan(want.g)  # [pages, H, S]
    mine = new_slot[:, 0]
    assert mine.sum().item() == sum(x for x, y in zip(new, own) if y is not None)
    keep = ~mine[:, None, :, None].expand_as(c.k)
    assert torch.equal(bits(c.k)[keep], bits(before[0])[keep])
    assert torch.equal(bits(c.g)[~new_slot], bits(before[2])[~new_slot])
    fresh = torch.isnan(before[3]) & ~torch.isnan(want.gbase)
    assert torch.equal(bits(c.gbase)[~fresh], bits(before[3])[~fresh])
    half = torch.finfo(c.dt).eps / 2

    def near_rotated(got, src, pos):
        from cachetest import rotate

        if not rot:
            return torch.equal(bits(got), bits(src))
        ref = rotate(src, cos[pos], sin[pos], pairs)
        top = src.double().abs().amax(-1, keepdim=True)
        return bool(((got.double() - ref).abs() <= half * ref.abs() * (1 + 2**-20) + 6 * top * 2.0**-24).all())

    for b in range(c.B):
        if own[b] is None:
            if rot:  # an idle sequence's rows are not written
                assert torch.isnan(out[c.row0[b] : c.row0[b] + new[b]]).all()
            continue
        p = torch.arange(own[b] - new[b], own[b], device="cuda")
        page = c.table[b].long()[p // S]
        assert near_rotated(c.k[page, :, p % S], c.seq[b][0][own[b] - new[b] :], c.P + p)
        if rot:
            r = slice(c.row0[b], c.row0[b] + new[b])
            assert near_rotated(out[r], c.q[r], c.P + p)
    if rot and c.rows > sum(new):
        assert torch.isnan(out[sum(new) :]).all()  # rows behind the last sequence
    tol = (8 + 11) * 2.0**-24
    got, ref = c.g.double()[new_slot], want.g.double()[new_slot]
    assert ((got - ref).abs() <= (tol + 2**-24) * ref.abs()).all()  # the reference's g is itself rounded
    got, ref = c.gbase.double().sum(-1), want.gbase.double().sum(-1)
    sel = fresh[..., 0]
    assert ((got - ref).abs()[sel] <= (tol + 2**-23) * ref.abs()[sel]).all()
    assert ((c.gbase[..., 1].abs() <= 2.0**-24 * c.gbase[..., 0].abs()) | ~sel).all()  # high holds all it can


def test_appending_token_by_token_gives_the_sums_of_one_append(fox):
    """150 tokens one at a time, in blocks of 13, and at once: the same K and V, gates within one addition a call."""
    own, S = 150, 32
    pools = []
    for block in (1, 13, 150):
        c = Case([own], [own], 4, 2, 64, S, seed=5)
        k, v, z = c.new_rows()
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        for t in range(0, own, block):
            m = min(block, own - t)
            c.lens.fill_(t + m)
            c.cu.copy_(torch.tensor([0, m], dtype=torch.int32))
            fox.fox_cache_append(c.cache(fox), c.batch(fox, max_new=m), k[t : t + m], v[t : t + m], z[t : t + m], ws=ws)
        assert fox.fox_check_error(ws) == 0
        pools.append(c)
    want = Case([own], [own], 4, 2, 64, S, seed=5)
    want.put()
    for c, adds in zip(pools, (S, 11 + S // 13 + 1, 11)):
        assert torch.equal(bits(c.k), bits(want.k)) and torch.equal(bits(c.v), bits(want.v))
        ok = ~torch.isnan(want.g)
        assert torch.equal(ok, ~torch.isnan(c.g))
        assert ((c.g - want.g).double().abs()[ok] <= (8 + adds + 2) * 2.0**-24 * want.g.double().abs()[ok]).all()
        a, b = c.gbase.double().sum(-1), want.gbase.double().sum(-1)
        ok = ~torch.isnan(b)
        assert torch.equal(ok, ~torch.isnan(a))
        assert ((a - b).abs()[ok] <= (8 + adds + 2) * 2.0**-24 * b.abs()[ok]).all()


def test_gates_at_the_ends_of_their_range(fox):
    """z = +inf is a gate that never closes (log 0 exactly); -80 takes 80 off; both beside ordinary ones."""
    c = Case([40], [40], 3, 1, 64, 16, seed=8)
    z = c.seq[0][2]
    z[:, 0] = float("inf")
    z[:, 1] = -80.0
    k, v, z = c.new_rows()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fox.fox_cache_append(c.cache(fox), c.batch(fox), k, v, z, ws=ws)
    t = c.table[0, :3].long()
    assert (c.g[t[0], 0] == 0).all() and (c.gbase[t, 0] == 0).all()
    assert c.g[t[0], 1].tolist() == [-80.0 * (i + 1) for i in range(16)]
    assert c.gbase[t, 1, 0].tolist() == [0.0, -1280.0, -2560.0]
    o, lse = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode gate ends")
    assert (lse.double() - rl).abs().max() <= foxtest.TOL_LSE_BF16


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
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", range(len(DECODES)))
def test_decode(fox, n, dtype):
    own, new, H, Hkv, d, S, more = DECODES[n]
    more = dict(more)
    bj, scale = more.pop("bias_from_j", False), more.pop("scale", None)
    c = Case(own, new, H, Hkv, d, S, dtype=dtype, seed=50 + n, **more)
    c.put()
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF  # nothing is read that the call has not written
    o, lse = torch.full_like(c.q, float("nan")), torch.full((c.rows, H), float("nan"), device="cuda")
    fox.fox_decode(cache, batch, c.q, scale=scale or 0.0, bias_from_j=bj, o=o, lse=lse, ws=ws)
    assert fox.fox_check_error(ws) == 0
    last = sum(new)
    assert torch.isnan(o[last:]).all() and torch.isnan(lse[last:]).all()
    ro, rl = c.attend(bias_from_j=bj, scale=scale)
    idle = torch.isinf(rl[:last])
    assert torch.equal(idle, torch.isinf(lse[:last])) and (o[:last][idle] == 0).all()
    if last:
        assert_o(tensor_f64(o[:last]), tensor_f64(ro[:last]), dtype, f"decode {n} {dtype}")
    if (~idle).any():
        tol = foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32
        assert (lse[:last].double() - rl[:last])[~idle].abs().max().item() <= tol
    # the same rows from a strided q, bit for bit
    wide = torch.cat([c.q.flatten(1), c.q.flatten(1)], 1)[:, H * d :].unflatten(1, (H, d))
    o2, lse2 = fox.fox_decode(cache, batch, wide, scale=scale or 0.0, bias_from_j=bj, ws=ws)
    assert torch.equal(bits(o2[:last]), bits(o[:last])) and torch.equal(bits(lse2[:last]), bits(lse[:last]))


# Behind prefixes long enough for the batch that they are shared out (one kernel for all sequences).
SHARED = [
    ([13, 1], [1, 1], 8, 8, 128, 64, 13001, dict(uniform=True, bias_from_j=True)),       # one row tile, keys split
    ([3] * 40, [1] * 40, 4, 1, 128, 16, 5003, dict(uniform=True)),                        # two row tiles
    ([20 + i % 3 for i in range(70)], [2] * 70, 12, 4, 64, 64, 1537, dict(tail=3)),       # five, a tail of one key
    ([None if i % 5 == 2 else 6 + 11 * (i % 4) for i in range(64)], [1 + i % 5 for i in range(64)], 14, 2, 128, 32, 1664,
     dict(tail=1)),                                                                       # odd group, idle ones, no tail
    ([9] * 9, [1] * 9, 20, 1, 128, 128, 22001, dict(uniform=True, scale=0.2)),            # a group of two head chunks
    ([40, 5, 77, 300], [33, 5, 40, 1], 6, 2, 64, 16, 10002, dict(bias_from_j=True)),      # many new tokens
]


@pytest.mark.parametrize("n", range(len(SHARED)))
def test_decode_behind_a_shared_prefix(fox, n):
    own, new, H, Hkv, d, S, P, more = SHARED[n]
    more = dict(more)
    bj, scale = more.pop("bias_from_j", False), more.pop("scale", None)
    c = Case(own, new, H, Hkv, d, S, seed=150 + n, prefix=P, **more)
    c.put()
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF
    o, lse = torch.full_like(c.q, float("nan")), torch.full((c.rows, H), float("nan"), device="cuda")
    fox.trace_begin()
    fox.fox_decode(cache, batch, c.q, scale=scale or 0.0, bias_from_j=bj, o=o, lse=lse, ws=ws)
    assert "prefix" in [k for k, _ in fox.trace_end()]
    assert fox.fox_check_error(ws) == 0
    last = sum(new)
    assert torch.isnan(o[last:]).all() and torch.isnan(lse[last:]).all()
    ro, rl = c.attend(bias_from_j=bj, scale=scale)
    idle = torch.isinf(rl[:last])
    assert torch.equal(idle, torch.isinf(lse[:last])) and (o[:last][idle] == 0).all()
    assert_o(tensor_f64(o[:last]), tensor_f64(ro[:last]), "bf16", f"decode shared {n}")
    assert (lse[:last].double() - rl[:last])[~idle].abs().max().item() <= foxtest.TOL_LSE_BF16
    o2, lse2 = fox.fox_decode(cache, batch, c.q, scale=scale or 0.0, bias_from_j=bj, ws=ws)
    assert torch.equal(bits(o2[:last]), bits(o[:last])) and torch.equal(bits(lse2[:last]), bits(lse[:last]))


@pytest.mark.parametrize("own,H,Hkv,d,S,P", [
    ([3, 70], 8, 2, 128, 64, 50001),            # one row tile: the streams share the keys out
    ([3] * 40, 4, 1, 64, 16, 12003),            # two row tiles
    ([5] * 90, 16, 4, 128, 128, 5000),          # three, the last item's second missing
])
def test_scores_that_rise_towards_the_prefix_s_start(fox, own, H, Hkv, d, S, P):
    """The prefix's keys are taken from the last on: here the row maximum is passed over and over, in every part."""
    c = Case(own, [1] * len(own), H, Hkv, d, S, prefix=P, uniform=True, seed=77, z_mean=9.0)
    k, v, z = c.pre
    grow = 1 + 12 * (1 - torch.arange(P, device="cuda") / P)
    c.pre = ((k.float() * grow[:, None, None]).to(k.dtype), v, z + 9)
    c.put()
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    o, lse = fox.fox_decode(cache, batch, c.q, ws=ws)
    assert fox.fox_check_error(ws) == 0
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode rising scores")
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


def test_many_small_weights_of_a_shared_prefix_count(fox):
    """One key of weight 1 and 400000 of 2^-26 whose values agree: O is 0.6 by these alone. Weights in fp16 that go down
    to 2^-35 are off by 2^-10 of themselves at 2^-26, and O is rounded by 2^-9 of itself: 2e-3."""
    P, d = 400000, 64
    c = Case([1, 1], [1, 1], 1, 1, d, 128, prefix=P, uniform=True, seed=5)
    k, v, z = c.pre
    k.zero_()
    k[P // 3] = 2.25  # a score of 18 = 64 * 2.25 / 8 against q of ones; 18 log2 e = 25.97
    v.fill_(100.0)
    v[P // 3] = 0.0
    z.fill_(float("inf"))
    c.q.fill_(1.0)
    for own in c.seq:
        own[0].zero_()
        own[1].zero_()
    c.put()
    o, lse = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert 0.3 < ro.min().item() and ro.max().item() < 0.7
    assert (o.double() - ro).abs().max().item() <= 2e-3
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


@pytest.mark.parametrize("B,P", [(3, 100), (40, 5003)])
def test_bad_pages_of_a_prefix_are_reported(fox, B, P):
    """Page ids of the prefix outside the pool: reported, read as page 0 (finite here), nothing else."""
    c = Case([9] * B, [1] * B, 4, 1, 128, 16, uniform=True, prefix=P, seed=6)
    c.put()
    for t in (c.k, c.v, c.g, c.gbase):
        t.nan_to_num_(0.0)
    c.ptable[1], c.ptable[2] = c.k.shape[0], -1
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    fox.fox_decode(cache, batch, c.q, ws=ws)
    assert fox.fox_check_error(ws) == FOX_ERR_DEVICE
    assert fox.fox_check_error(ws) == 0


def test_shared_values_outside_fp16_are_reported(fox):
    """The shared prefix's P V runs in fp16, like fox_fwd's: a V of 65536 or more there sets the error word; the
    same value among a sequence's own tokens, or in a prefix that is walked, is no error."""
    for B, P, status in ((40, 5003, FOX_ERR_DEVICE), (3, 100, 0)):
        for where in ("prefix", "own"):
            c = Case([9] * B, [1] * B, 4, 1, 128, 16, uniform=True, prefix=P, seed=6)
            (c.pre if where == "prefix" else c.seq[1])[1][5, 0, 7] = 1.0e6
            c.put()
            cache, batch = c.cache(fox), c.batch(fox)
            ws = fox.cache_workspace(cache, batch, c.rows)
            fox.fox_decode(cache, batch, c.q, ws=ws)
            assert fox.fox_check_error(ws) == (status if where == "prefix" else 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("own,new,H,Hkv,d,prefix", [
    ([70001], [1], 4, 1, 128, 0), ([30011, 5, 9000], [1, 3, 2], 8, 2, 64, 0), ([11], [1], 16, 16, 64, 20000),
    ([7, 130], [8 - 1, 6], 8, 2, 128, 9999)])
def test_decode_long_contexts_are_split_and_joined(fox, dtype, own, new, H, Hkv, d, prefix):
    c = Case(own, new, H, Hkv, d, 64, dtype=dtype, seed=77, prefix=prefix)
    c.put()
    o, lse = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), dtype, f"decode long {own[0]} {dtype}")
    assert (lse.double() - rl).abs().max().item() <= (foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32)


def test_decode_of_many_sequences(fox):
    own = [(b * 37) % 90 + 1 if b % 11 else None for b in range(600)]
    c = Case(own, [1] * 600, 8, 4, 64, 16, uniform=True, seed=9)
    c.put()
    o, lse = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode many")
    live = ~torch.isinf(rl)
    assert (lse.double() - rl)[live].abs().max().item() <= foxtest.TOL_LSE_BF16 and torch.isinf(lse[~live]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d,S", [(16, 64, 16), (9, 128, 32)])
def test_decode_of_the_most_sequences(fox, dtype, H, d, S):
    """2048 of them, in the widest row tile: the most shared memory that a call takes."""
    own = [b % 35 + 1 if b % 7 else None for b in range(2048)]
    c = Case(own, [1] * 2048, H, 1, d, S, dtype=dtype, uniform=True, seed=10)
    c.put()
    o, lse = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), dtype, "decode most")
    live = ~torch.isinf(rl)
    tol = foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32
    assert (lse.double() - rl)[live].abs().max().item() <= tol and torch.isinf(lse[~live]).all()


@pytest.mark.parametrize("prefix", [0, 40])
def test_pages_beyond_32_bit_offsets(fox, prefix):
    """A pool of 2^31 elements and more, the pages in use at its end."""
    pages = (1 << 31) // (8 * 128 * 128) + 40
    c = Case([300, 17], [2, 17], 16, 8, 128, 128, pages=pages, prefix=prefix, seed=4)
    c.put(upto_new=False)
    k, v, z = c.new_rows()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cache, batch = c.cache(fox), c.batch(fox)
    fox.fox_cache_append(cache, batch, k, v, z, ws=ws)
    o, lse = fox.fox_decode(cache, batch, c.q)
    assert fox.fox_check_error(ws) == 0
    ro, rl = c.attend()
    assert_o(tensor_f64(o), tensor_f64(ro), "bf16", "decode far pages")
    assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 100])
def test_what_the_batch_cannot_hold_is_reported_and_skipped(fox, dtype, prefix):
    """Bad page ids, lengths and row ranges: the bounds checks report them, nothing else changes."""
    own, new = [40, 70, 33], [2, 2, 2]

    def fresh():
        c = Case(own, new, 4, 2, 64, 16, dtype=dtype, seed=21, prefix=prefix)
        c.put(upto_new=False)
        return c

    good = fresh()
    k, v, z = good.new_rows()
    fox.fox_cache_append(good.cache(fox), good.batch(fox), k, v, z)
    o0, l0 = fox.fox_decode(good.cache(fox), good.batch(fox), good.q)
    ro, rl = good.attend()
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
        cache, batch = c.cache(fox), c.batch(fox)
        ws = fox.cache_workspace(cache, batch, c.rows)
        fox.fox_cache_append(cache, batch, k, v, z, ws=ws)
        assert fox.fox_check_error(ws) == FOX_ERR_DEVICE, what
        o, lse = fox.fox_decode(cache, batch, c.q, ws=ws)
        assert fox.fox_check_error(ws) == FOX_ERR_DEVICE, what
        assert fox.fox_check_error(ws) == 0
        rows = [0, 1] if what == "falling rows" else [0, 1, 4, 5]
        if "page" in what:
            assert torch.equal(bits(o[rows]), bits(o0[rows])) and torch.equal(bits(lse[rows]), bits(l0[rows])), what
        else:
            # A skipped sequence has no work, so the others' keys are split among the workers elsewhere and
            # their fp32 sums of at most 200 terms round elsewhere (each side within 200 * 2^-24 of the exact
            # sum, and LSE by as much): not the same bits, but within the bounds of the exact values.
            assert_o(tensor_f64(o[rows]), tensor_f64(ro[rows]), dtype, f"decode beside {what} {dtype}")
            assert (lse[rows].double() - rl[rows]).abs().max() <= (
                foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32), what
        ids = torch.cat([good.table[0, :3], good.table[2, :3]]) if what != "falling rows" else good.table[0, :3]
        for a, b in ((c.k, good.k), (c.v, good.v), (c.g, good.g), (c.gbase, good.gbase)):
            assert torch.equal(bits(a[ids.long()]), bits(b[ids.long()])), what


def test_positions_behind_the_tables_are_reported(fox):
    c = Case([40, 20], [1, 1], 4, 2, 64, 16, uniform=True, seed=3)
    c.put(upto_new=False)
    k, v, z = c.new_rows()
    cos, sin = angles(39, 64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    before = c.k.clone()
    fox.fox_cache_append(c.cache(fox), c.batch(fox), k, v, z, cos=cos, sin=sin, ws=ws)
    assert fox.fox_check_error(ws) == FOX_ERR_DEVICE
    assert torch.equal(bits(c.k[c.table[0].long()]), bits(before[c.table[0].long()]))


def test_binding_refusals(fox):
    c = Case([40, 20], [1, 1], 4, 2, 64, 16, uniform=True, seed=3)
    cache, batch = c.cache(fox), c.batch(fox)
    k, v, z = c.new_rows()
    for bad in (c.q[:, :2], c.q.transpose(0, 1), c.q[..., :32], c.q[:, :, ::2].repeat(1, 1, 2)[:, :, ::2]):
        with pytest.raises(ValueError):
            fox.fox_decode(cache, batch, bad)
    with pytest.raises(TypeError):
        fox.fox_decode(cache, batch, c.q.float())
    with pytest.raises(ValueError):
        fox.fox_decode(cache, batch, c.q.cpu())
    with pytest.raises(ValueError):
        fox.fox_decode(cache, batch, c.q, o=torch.empty(2, 4, 128, device="cuda", dtype=torch.bfloat16)[..., ::2])
    with pytest.raises(ValueError):
        fox.fox_decode(cache, batch, c.q, lse=torch.empty(4, 2, device="cuda").t())
    with pytest.raises(fox.FoxError):
        fox.fox_decode(cache, batch, c.q[:1])  # one row does not go around two sequences
    with pytest.raises(fox.FoxError):
        fox.fox_decode(cache, batch, c.q, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fox.fox_cache_append(cache, batch, k, v, z[:, :3])
    with pytest.raises(ValueError):
        fox.fox_cache_append(cache, batch, k, v[:1], z)
    with pytest.raises(ValueError):
        fox.fox_cache_append(cache, batch, k, v, z, q=c.q)
    cos, sin = angles(50, 64)
    with pytest.raises(ValueError):
        fox.fox_cache_append(cache, batch, k, v, z, cos=cos)
    with pytest.raises(ValueError):
        fox.fox_cache_append(cache, batch, k, v, z, cos=cos, sin=sin[:40])
    with pytest.raises(fox.FoxError):
        fox.fox_cache_append(cache, batch, k, v, z, *(), cos=cos[:, :12].contiguous(), sin=sin[:, :12].contiguous())
    with pytest.raises(ValueError):
        fox.make_cache(c.k.transpose(0, 1), c.v, c.g, c.gbase)
    with pytest.raises(ValueError):
        fox.make_batch(c.lens, c.table.t().contiguous().t())


# ------------------------------------------------------------------------------------ in use


@pytest.mark.parametrize("d,S,bias_from_j", [(128, 64, False), (64, 16, True)])
def test_prompt_then_tokens_as_the_forward_sees_them(fox, d, S, bias_from_j):
    """A prompt through fox_fwd and into the cache, then tokens one at a time and three at a time: every
    row is the forward's over the whole sequence."""
    B, N0, N, H = 3, 150, 190, 4
    gen = torch.Generator("cuda").manual_seed(11)
    q, k, v = (torch.randn(B, N, H, d, generator=gen, device="cuda").bfloat16() for _ in range(3))
    z = torch.randn(B, N, H, generator=gen, device="cuda") + torch.linspace(0, 5, H, device="cuda")
    full_o, full_l = fox.fox_fwd(q, k, v, z, bias_from_j=bias_from_j)
    width = -(-N // S)
    cache = fox.new_cache(B * width + 1, S, H, H, d)
    table = torch.randperm(B * width + 1, device="cuda")[: B * width].view(B, width).to(torch.int32)
    lens = torch.full((B,), N0, dtype=torch.int32, device="cuda")
    batch = fox.make_batch(lens, table, max_new=N0)
    rows = lambda x, t0, t1: x[:, t0:t1].reshape(B * (t1 - t0), *x.shape[2:])  # noqa: E731
    ws = fox.cache_workspace(cache, batch, B * N0)
    fox.fox_cache_append(cache, batch, rows(k, 0, N0), rows(v, 0, N0), rows(z, 0, N0), ws=ws)
    t = N0
    while t < N:
        m = min(3 if t % 2 else 1, N - t)
        lens.fill_(t + m)
        fox.fox_cache_append(cache, batch, rows(k, t, t + m), rows(v, t, t + m), rows(z, t, t + m), ws=ws)
        o, lse = fox.fox_decode(cache, batch, rows(q, t, t + m), bias_from_j=bias_from_j, ws=ws)
        # both are within the bound of the same exact values, so within twice of each other
        ref_o, ref_l = rows(full_o, t, t + m), rows(full_l, t, t + m)
        big = torch.maximum(o.float().abs(), ref_o.float().abs()) >= 4
        assert ((o.float() - ref_o.float()).abs()[~big] <= 2 * foxtest.TOL_O_BF16).all()
        assert ((o.float() - ref_o.float()).abs()[big] <= 2.0**-5).all()
        assert (lse - ref_l).abs().max() <= 2 * foxtest.TOL_LSE_BF16
        t += m
    assert fox.fox_check_error(ws) == 0


@pytest.mark.parametrize("P", [200, 25001])
def test_a_shared_prefix_gives_what_copies_of_it_give(fox, P):
    """Sequences behind one shared prefix, and the same sequences each with the prefix's tokens of its own."""
    own, H, Hkv, d, S = [40, 1, 17, 90], 8, 2, 128, 32
    c = Case(own, [1] * 4, H, Hkv, d, S, prefix=P, uniform=True, seed=14)
    c.put()
    o, lse = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    full = Case([P + x for x in own], [1] * 4, H, Hkv, d, S, uniform=True, seed=15)
    for b in range(4):
        full.seq[b] = tuple(torch.cat([x, y]) for x, y in zip(c.pre, c.seq[b]))
    full.put()
    o2, lse2 = fox.fox_decode(full.cache(fox), full.batch(fox), c.q)
    ro, rl = c.attend()
    for a, l, name in ((o, lse, "shared"), (o2, lse2, "own copies")):
        assert_o(tensor_f64(a), tensor_f64(ro), "bf16", f"decode prefix {name}")
        assert (l.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix,B", [(0, 5), (130, 5), (300, 40), (7000, 40)])
def test_captured_steps_replay_on_new_contents(fox, dtype, prefix, B):
    """Append and decode captured once and replayed while the lengths grow: bit for bit the eager calls."""
    H, Hkv, d, S, first, steps = 8, 2, 64, 16, 30, 5
    own = [first + 3 * (b % 7) + steps if b != 2 else None for b in range(B)]
    c = Case(own, [1] * B, H, Hkv, d, S, dtype=dtype, uniform=True, prefix=prefix, seed=31)
    e = Case(own, [1] * B, H, Hkv, d, S, dtype=dtype, uniform=True, prefix=prefix, seed=31)
    cos, sin = angles(prefix + 120, d)
    toks = [c.seq[b] for b in range(B)]
    live = c.lens > 0
    for x in (c, e):
        x.lens -= steps * live
        x.own = [None if y is None else y - steps for y in own]
        x.put()
    k, v = (torch.zeros(B, Hkv, d, device="cuda", dtype=c.dt) for _ in range(2))
    z, q = torch.zeros(B, H, device="cuda"), c.q.clone()
    o, lse, qr = torch.empty_like(q), torch.empty(B, H, device="cuda"), torch.empty_like(q)
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, B)
    ws2 = fox.cache_workspace(cache, batch, B)

    def step(cache, batch, o, lse, ws):
        fox.fox_cache_append(cache, batch, k, v, z, q=q, cos=cos, sin=sin, q_out=qr, ws=ws)
        fox.fox_decode(cache, batch, qr, o=o, lse=lse, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(cache, batch, o, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    eo, el = torch.empty_like(o), torch.empty_like(lse)
    for t in range(steps):
        for b in range(B):
            if own[b] is None:
                continue
            for dst, src in zip((k, v, z), toks[b]):
                dst[b] = src[own[b] - steps + t]
        q.normal_(generator=c.gen)
        c.lens += live.int()
        e.lens += live.int()
        graph.replay()
        step(e.cache(fox), e.batch(fox), eo, el, ws2)
        assert torch.equal(bits(o), bits(eo)) and torch.equal(bits(lse), bits(el)), t
        for a, b in ((c.k, e.k), (c.v, e.v), (c.g, e.g), (c.gbase, e.gbase)):
            assert torch.equal(bits(a), bits(b)), t
    assert fox.fox_check_error(ws) == 0 and fox.fox_check_error(ws2) == 0


@pytest.mark.parametrize("prefix", [0, 26000])
def test_captured_calls_behind_a_fork_and_a_join(fox, prefix):
    """In a graph: k and v made on one stream, z on another, append behind both, two decodes side by side."""
    H, Hkv, d, S, nan = 8, 2, 128, 64, float("nan")
    c = Case([70, 300], [1, 1], H, Hkv, d, S, uniform=True, prefix=prefix, seed=32)
    c.put()
    want = fox.fox_decode(c.cache(fox), c.batch(fox), c.q)
    k0, v0, z0 = c.new_rows()
    for b in range(2):  # the new tokens out of the cache again
        page, slot = int(c.table[b, (c.own[b] - 1) // S]), (c.own[b] - 1) % S
        c.k[page, :, slot] = nan
        c.v[page, :, slot] = nan
        c.g[page, :, slot] = nan
    k, v, z = torch.zeros_like(k0), torch.zeros_like(v0), torch.zeros_like(z0)
    outs = [(torch.empty_like(c.q), torch.empty(2, H, device="cuda")) for _ in range(2)]
    cache, batch = c.cache(fox), c.batch(fox)
    ws = [fox.cache_workspace(cache, batch, 2) for _ in range(2)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z.copy_(z0)
            z.mul_(1.0)
        k.copy_(k0)
        v.copy_(v0)
        main.wait_stream(side)
        fox.fox_cache_append(cache, batch, k, v, z, ws=ws[0])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            fox.fox_decode(cache, batch, c.q, o=outs[1][0], lse=outs[1][1], ws=ws[1])
        fox.fox_decode(cache, batch, c.q, o=outs[0][0], lse=outs[0][1], ws=ws[0])
        main.wait_stream(side)
    for _ in range(3):
        for o, lse in outs:
            o.fill_(nan)
            lse.fill_(nan)
        k.fill_(nan)
        z.fill_(nan)
        graph.replay()
        torch.cuda.synchronize()
        for o, lse in outs:
            assert torch.equal(bits(o), bits(outs[0][0])) and torch.equal(bits(lse), bits(outs[0][1]))
            # The new token's g is one fp32 sum here, rounded from 64 bits there: below 128, so 2^-17 apart and
            # some ulps of log sigmoid; O may then round to the neighbouring value.
            assert (lse - want[1]).abs().max() <= 2.0**-15
            x, y = o.float(), want[0].float()
            assert ((x - y).abs() <= 2.0**-7 * torch.maximum(x.abs(), y.abs()) + 2.0**-15).all()
    assert fox.fox_check_error(ws[0]) == 0 and fox.fox_check_error(ws[1]) == 0


def test_calls_on_another_stream_and_two_at_once(fox):
    cases = [Case([3000, 50], [1, 1], 8, 2, 128, 64, uniform=True, seed=s, prefix=p) for s, p in ((1, 0), (2, 500), (3, 26000))]
    want = []
    for c in cases:
        c.put()
        want.append(fox.fox_decode(c.cache(fox), c.batch(fox), c.q))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in cases]
    for _ in range(4):
        for n, c in enumerate(cases):
            got[n].append(fox.fox_decode(c.cache(fox), c.batch(fox), c.q, stream=streams[n]))
    torch.cuda.synchronize()
    for n, (o, lse) in enumerate(want):
        for a, b in got[n]:
            assert torch.equal(bits(a), bits(o)) and torch.equal(bits(b), bits(lse))


def test_back_to_back_calls_on_one_workspace(fox):
    cases = [Case(own, [1] * len(own), 8, 2, 128, 64, uniform=True, seed=40 + i, prefix=p)
             for i, (own, p) in enumerate([([900] * 3, 0), ([10] * 3, 40000), ([2000, 1, 1], 0), ([10] * 3, 700)])]
    for c in cases:
        c.put()
    hs = [(c.cache(fox), c.batch(fox), c.q) for c in cases]
    size = max(fox.fox_cache_workspace_bytes(a, b, 3) for a, b, _ in hs)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = [fox.fox_decode(*h) for h in hs]
    torch.cuda.synchronize()
    got = [[fox.fox_decode(*h, ws=ws) for h in hs] for _ in range(4)]
    torch.cuda.synchronize()
    for round_ in got:
        for (o, lse), (o0, l0) in zip(round_, want):
            assert torch.equal(bits(o), bits(o0)) and torch.equal(bits(lse), bits(l0))
    assert fox.fox_check_error(ws) == 0
