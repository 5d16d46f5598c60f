"""Pages of the pool on the GPU against the definition (pagestest.py): whole numbers, equal. And the copies that go with
them: pages bit for bit."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FOX_ERR_DEVICE = 6
MARK = -77  # in what nothing writes


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    fox.lib()
    return fox


def ints(x, *shape):
    t = torch.tensor(x, dtype=torch.int32, device="cuda")
    return t.view(*shape) if shape else t


class Pool:
    """Sequences on a pool, some of which share pages, made at random."""

    def __init__(self, rng, B, S, stride, pages, prefix=0, share=0.3, idle=0.1, full=1.0):
        self.S, self.stride, self.P, self.N, self.B = S, stride, prefix, pages, B
        order = rng.sample(range(pages), pages)
        npre = -(-prefix // S)
        self.prefix_table = [order.pop() for _ in range(npre)]
        self.lens, self.table = [], []
        for b in range(B):
            row = [MARK] * stride
            if rng.random() < idle:
                own = 0
                self.lens.append(0)
            elif b and rng.random() < share and any(self.lens):
                root = rng.choice([i for i in range(b) if self.lens[i]])
                root_own = self.lens[root] - prefix
                same = rng.random() < 0.5
                own = root_own if same else rng.randint(0, max(0, int(stride * S * full)))
                shared = -(-own // S) if same else min(rng.randint(0, root_own), own) // S
                row[:shared] = self.table[root][:shared]
                need = -(-own // S) - shared
                if need > len(order):
                    own, need = shared * S, 0
                row[shared : shared + need] = [order.pop() for _ in range(need)]
                self.lens.append(prefix + own)
            else:
                own = rng.randint(0, int(stride * S * full))
                need = -(-own // S)
                if need > len(order):
                    own, need = 0, 0
                row[:need] = [order.pop() for _ in range(need)]
                self.lens.append(prefix + own)
            if self.lens[-1] == prefix and prefix == 0:
                self.lens[-1] = 0
            self.table.append(row)
        self.refs = [0] * pages
        for i in self.prefix_table:
            self.refs[i] += 1
        for b in range(B):
            if self.lens[b]:
                for c in range(-(-(self.lens[b] - prefix) // S)):
                    self.refs[self.table[b][c]] += 1

    def pages(self, fox, refs=None, lens=None, table=None, prefix_table=None):
        pre = ints(self.prefix_table) if self.P else None
        return fox.make_pages(self.S, ints(self.refs) if refs is None else refs, ints(self.lens) if lens is None else lens,
                              ints(self.table, self.B, self.stride) if table is None else table,
                              prefix_table=pre if prefix_table is None else prefix_table, prefix_len=self.P)

    def blank(self, fox, B):
        full = lambda *s: torch.full(s, MARK, dtype=torch.int32, device="cuda")  # noqa: E731
        return fox.make_pages(self.S, full(self.N), full(B), full(B, self.stride),
                              prefix_table=full(len(self.prefix_table)) if self.P else None, prefix_len=self.P)


def table_of(rows, B, stride, start=None):
    t = [[MARK] * stride for _ in range(B)] if start is None else [list(r) for r in start]
    for (b, c), page in rows.items():
        t[b][c] = page
    return t


# B, S, stride, pages, prefix, new B, largest add
STEPS = [
    (1, 16, 4, 40, 0, 1, 3), (3, 16, 1, 3, 0, 5, 16), (8, 64, 16, 200, 0, 8, 1), (8, 128, 5, 12, 300, 8, 200),
    (40, 32, 9, 300, 0, 64, 5), (100, 16, 30, 2000, 17, 70, 1), (500, 64, 20, 9000, 0, 500, 130), (2048, 16, 3, 5000, 0, 2048, 2),
    (1100, 16, 8, 1400, 5, 1100, 40), (7, 16, 3000, 30000, 0, 9, 9000), (5, 16, 2, 1, 0, 5, 1), (64, 64, 4, 100000, 0, 64, 64),
]


@pytest.mark.parametrize("n", range(len(STEPS)))
@pytest.mark.parametrize("how", ["branches", "go on", "in place"])
def test_step(fox, n, how):
    import pagestest

    B, S, stride, N, P, B2, most = STEPS[n]
    rng = random.Random(100 + n)
    x = Pool(rng, B, S, stride, N, P, full=rng.choice([0.3, 0.9, 1.0]))
    if how == "branches":
        parent = [rng.choice([-1, rng.randrange(B), rng.randrange(B), min(b, B - 1)]) for b in range(B2)]
    else:
        B2, parent = B, list(range(B))
    add = [rng.choice([0, 1, 1, rng.randint(0, most)]) for _ in range(B2)]
    # without parent an idle sequence begins where it stands
    refs, lens, rows, copies, short = pagestest.step(x.refs, x.lens, x.table, parent, add, S, P, B2)
    now = x.pages(fox)
    out = now if how == "in place" else x.blank(fox, B2)
    got = torch.full((B2, 2), MARK, dtype=torch.int32, device="cuda")
    ws = fox.pages_workspace(now, out)
    ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF
    for _ in range(1 if how == "in place" else 3):  # the same again from the same
        fox.fox_pages_step(now, ints(add), got, parent=ints(parent) if how == "branches" else None,
                           out=None if how == "in place" else out, ws=ws)
        assert fox.fox_check_error(ws) == (FOX_ERR_DEVICE if short else 0)
    assert out.refs.tolist() == refs
    assert out.lens.tolist() == lens
    assert out.table.tolist() == table_of(rows, B2, stride, x.table if how == "in place" else None)
    assert [tuple(c) for c in got.tolist()] == copies
    # every page in use is named as often as refs says
    for b in range(B2):
        for c in range(pagestest.pages_of(lens[b] - P if lens[b] else 0, S)):
            refs[rows[b, c] if (b, c) in rows else x.table[b][c]] -= 1
    for i in x.prefix_table:
        refs[i] -= 1
    assert not any(refs)


@pytest.mark.parametrize("stride", [500, 1000])  # references counted by the step itself, and by a kernel of their own
def test_most_sequences_go_on_from_one(fox, stride):
    import pagestest

    x = Pool(random.Random(9), 3, 16, stride, 8000, 0, full=0.5, idle=0)
    parent, add = [1] * 2047 + [2], [1] * 2048
    refs, lens, rows, copies, short = pagestest.step(x.refs, x.lens, x.table, parent, add, 16, 0, 2048)
    now, out = x.pages(fox), x.blank(fox, 2048)
    got, ws = ints([0] * 4096, 2048, 2), fox.pages_workspace(now, out)
    fox.fox_pages_step(now, ints(add), got, parent=ints(parent), out=out, ws=ws)
    assert not short and fox.fox_check_error(ws) == 0
    assert out.refs.tolist() == refs and out.lens.tolist() == lens
    assert out.table.tolist() == table_of(rows, 2048, stride) and [tuple(c) for c in got.tolist()] == copies


def test_step_of_what_does_not_fit_is_reported(fox):
    """Parents, lengths, adds and pages outside their ranges: reported, the other sequences as if it were not there."""
    import pagestest

    for what in ("parent", "length", "negative length", "add", "page", "inside the prefix"):
        rng = random.Random(5)
        x = Pool(rng, 6, 16, 8, 100, 40, idle=0, share=0)
        parent, add = list(range(6)), [3] * 6
        given, given_parent, given_add = x, list(parent), list(add)
        lens, table = list(x.lens), [list(r) for r in x.table]
        x.lens[2] = x.P + 37  # two pages and a part
        if what == "parent":
            given_parent[2], parent[2] = 6, -1
        elif what == "length":
            x.lens[2], lens[2] = x.P + 8 * 16 + 1, 0
        elif what == "negative length":
            x.lens[2], lens[2] = -1, 0
        elif what == "inside the prefix":
            x.lens[2], lens[2] = x.P - 1, 0
        elif what == "add":
            given_add[2], add[2] = -3, 0
            lens[2] = x.lens[2]
        else:
            x.lens[2] = lens[2] = x.P + 37
            given_parent = parent = [0, 1, -1, 3, 4, 5]
            table[2][1] = x.table[2][1] = 100
        x = Pool.__new__(Pool)
        x.__dict__.update(given.__dict__)
        now, out = x.pages(fox), x.blank(fox, 6)
        got = torch.full((6, 2), MARK, dtype=torch.int32, device="cuda")
        ws = fox.pages_workspace(now, out)
        fox.fox_pages_step(now, ints(given_add), got, parent=ints(given_parent), out=out, ws=ws)
        assert fox.fox_check_error(ws) == FOX_ERR_DEVICE, what
        assert fox.fox_check_error(ws) == 0
        if what == "page":
            continue
        if what == "parent":
            lens = list(x.lens)
        refs, want, rows, copies, short = pagestest.step(x.refs, lens, table, parent, add, 16, x.P, 6)
        assert out.lens.tolist() == want, what
        keep = [b for b in range(6) if b != 2]
        t = table_of(rows, 6, 8)
        assert [out.table.tolist()[b] for b in keep] == [t[b] for b in keep], what


@pytest.mark.parametrize("n", range(9))
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(fox, n, in_place):
    import pagestest

    B, S, stride, N, P, most = [(1, 16, 4, 40, 0, 50), (0, 16, 4, 17, 0, 5), (5, 16, 3, 16, 0, 16), (60, 32, 9, 1500, 100, 1000),
                                (60, 32, 9, 1500, 100, 37), (2048, 16, 3, 9000, 0, 9000), (300, 64, 30, 20000, 64, 0),
                                (40, 16, 500, 70000, 3, 1 << 17), (3, 128, 2, 5, 0, 3)][n]
    x = Pool(random.Random(200 + n), B, S, stride, N, P, idle=0.3)
    refs, rows, prefix, new, moves, used = pagestest.compact(x.refs, x.lens, x.table, x.prefix_table, S, P, most)
    now = x.pages(fox) if B else fox.make_pages(S, ints(x.refs), ints([]), torch.zeros(0, stride, dtype=torch.int32, device="cuda"))
    lens = now.lens.clone()
    out = now if in_place else x.blank(fox, B)
    full = lambda *s: torch.full(s, MARK, dtype=torch.int32, device="cuda")  # noqa: E731
    gmap, gmoves, gused = full(N), full(most, 2), full(2)
    ws = fox.pages_workspace(now, out)
    ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF
    for _ in range(1 if in_place else 3):
        fox.fox_pages_compact(now, gmap, gmoves, gused, out=None if in_place else out, ws=ws)
        assert fox.fox_check_error(ws) == 0
    assert out.refs.tolist() == refs
    assert gmap.tolist() == new and tuple(gused.tolist()) == used
    assert [tuple(m) for m in gmoves.tolist()] == (moves + [(-1, -1)] * most)[:most]
    if B:
        assert out.table.tolist() == table_of(rows, B, stride, x.table if in_place else None)
        assert torch.equal(now.lens, lens)
    if P:
        assert out.prefix_table.tolist() == prefix


def test_compact_reports_entries_outside_the_pool(fox):
    x = Pool(random.Random(9), 4, 16, 4, 60, 0, idle=0, share=0)
    x.lens[1] = 40
    x.table[1][:3] = [60, -1, 5]
    now, out = x.pages(fox), x.blank(fox, 4)
    ws = fox.pages_workspace(now, out)
    fox.fox_pages_compact(now, ints([0] * 60), ints([0] * 40, 20, 2), ints([0, 0]), out=out, ws=ws)
    assert fox.fox_check_error(ws) == FOX_ERR_DEVICE
    assert out.table[1, :2].tolist() == [60, -1]


def arrays(c):
    return [x for x in (c.k, c.v, getattr(c, "ks", None), getattr(c, "vs", None), c.g, c.gbase, c.g_low) if x is not None]


@pytest.mark.parametrize("kind", ["4bit", "bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,d,S,pages,n,low", [(1, 1, 64, 16, 7, 3, True), (14, 2, 128, 64, 60, 25, False), (9, 3, 64, 32, 300, 140, True),
                                                   (32, 8, 128, 128, 12, 6, True),
                                                   (9, 1, 64, 16, 1500, 700, True), (8, 2, 64, 16, 900, 400, False)])  # many small pages
def test_copy(fox, kind, H, Hkv, d, S, pages, n, low):
    gen = torch.Generator("cuda").manual_seed(1)
    c = (fox.new_cache4(pages, S, H, Hkv, d) if kind == "4bit" else
         fox.new_cache(pages, S, H, Hkv, d, dtype=torch.bfloat16 if kind == "bf16" else torch.float32))
    if not low:
        c = (fox.make_cache4(c.k, c.v, c.ks, c.vs, c.g, c.gbase) if kind == "4bit" else fox.make_cache(c.k, c.v, c.g, c.gbase))
    for x in arrays(c):  # any bits, NaN among them
        raw = x.view(torch.uint8) if x.dtype != torch.uint8 else x
        raw.copy_(torch.randint(0, 256, raw.shape, generator=gen, device="cuda", dtype=torch.uint8))
    order = torch.randperm(pages, generator=gen, device="cuda")
    pairs = torch.stack([order[:n], order[n : 2 * n]], 1).to(torch.int32)
    pairs = torch.cat([pairs[: n // 2], ints([[-1, -1]]), pairs[n // 2 :]]).contiguous()
    want = [x.clone() for x in arrays(c)]
    for x in want:
        x[order[n : 2 * n]] = x[order[:n]]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fox.fox_cache_copy(c, pairs, ws=ws)
    assert fox.fox_check_error(ws) == 0
    for x, y in zip(arrays(c), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # ids outside the pool: reported, nothing is copied for them
    bad = ints([[pages, int(order[0])], [int(order[0]), -1], [-5, -5], [int(order[0]), pages + 7]] * (300 if n >= 400 else 1))
    fox.fox_cache_copy(c, bad, ws=ws)
    assert fox.fox_check_error(ws) == FOX_ERR_DEVICE
    for x, y in zip(arrays(c), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    fox.fox_cache_copy(c, pairs[:0], ws=ws)


def test_copies_beyond_32_bit_offsets(fox):
    pages = (1 << 32) // (8 * 128 * 64) + 3
    c = fox.new_cache4(pages, 128, 8, 8, 128)
    pairs = ints([[pages - 1, 0], [1, pages - 2]])
    for x in arrays(c):
        for p in (0, 1, pages - 2, pages - 1):
            x[p] = p % 100
    fox.fox_cache_copy(c, pairs)
    for x in arrays(c):
        for p, q in ((0, pages - 1), (pages - 2, 1), (1, 1), (pages - 1, pages - 1)):
            assert (x[p] == q % 100).all()


@pytest.mark.parametrize("kind", ["4bit", "bf16"])
def test_a_search_over_a_cache(fox, kind):
    """Hypotheses that branch, end and go on, with pages handed out and copied step by step, and the pool packed on the way: at every
    step each attends to its own tokens, as a plain list of tokens has them."""
    import foxtest
    from cachetest import Case
    from foxtest import assert_o, tensor_f64
    from fourtest import hold

    H, Hkv, d, S, B, N, stride = 8, 2, 64, 16, 5, 60, 8
    rng, gen = random.Random(3), torch.Generator("cuda").manual_seed(3)
    cache = fox.new_cache4(N, S, H, Hkv, d) if kind == "4bit" else fox.new_cache(N, S, H, Hkv, d)
    append, decode = (fox.fox_cache4_append, fox.fox_cache4_decode) if kind == "4bit" else (fox.fox_cache_append, fox.fox_decode)
    zeros = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    refs, tabs, lens = ([zeros(*s) for _ in range(2)] for s in ((N,), (B, stride), (B,)))
    state = [fox.make_pages(S, refs[i], lens[i], tabs[i]) for i in range(2)]
    pws = fox.pages_workspace(*state)
    copies, now = zeros(B, 2), 0
    rnd = lambda n, *s: torch.randn(n, *s, generator=gen, device="cuda")  # noqa: E731
    empty = (rnd(0, Hkv, d).bfloat16(), rnd(0, Hkv, d).bfloat16(), rnd(0, H))
    said = [empty] * B
    for t in range(12):
        parent = list(range(B)) if t == 0 else [rng.randrange(B) if rng.random() < 0.4 else b for b in range(B)]
        add = [20 + b for b in range(B)] if t == 0 else [rng.choice([1, 1, 1, 7]) for _ in range(B)]
        if t == 6:
            parent[2], add[2] = -1, 0  # a place that stays idle
        fox.fox_pages_step(state[now], ints(add), copies, parent=ints(parent), out=state[1 - now], ws=pws)
        now = 1 - now
        fox.fox_cache_copy(cache, copies)
        if t in (4, 9):
            moves, used = zeros(N, 2), zeros(2)
            fox.fox_pages_compact(state[now], zeros(N), moves, used, ws=pws)
            fox.fox_cache_copy(cache, moves)
            in_use = int((refs[now] > 0).sum())
            assert used.tolist() == [in_use, in_use] and (refs[now][:in_use] > 0).all()
        assert fox.fox_check_error(pws) == 0
        new = [(rnd(n, Hkv, d).bfloat16(), rnd(n, Hkv, d).bfloat16(), rnd(n, H) + 3) for n in add]
        said = [tuple(torch.cat([x, y]) for x, y in zip(said[p] if p >= 0 else empty, y)) for p, y in zip(parent, new)]
        rows = [torch.cat([x[i] for x in new]) for i in range(3)]
        cu = ints([sum(add[:b]) for b in range(B + 1)])
        batch = fox.make_batch(lens[now], tabs[now], cu_new=cu, max_new=max(add))
        ws = (fox.cache4_workspace if kind == "4bit" else fox.cache_workspace)(cache, batch, sum(add))
        append(cache, batch, *rows, ws=ws)
        q = rnd(sum(add), H, d).bfloat16()
        o, lse = decode(cache, batch, q, ws=ws)
        assert fox.fox_check_error(ws) == 0
        c = Case([x[0].shape[0] or None for x in said], add, H, Hkv, d, S, seed=1)
        c.seq = [((hold(x[0])[2], hold(x[1])[2], x[2]) if kind == "4bit" else x) for x in said]
        c.q = q
        ro, rl = c.attend()
        assert_o(tensor_f64(o), tensor_f64(ro), "bf16", f"search {kind}")
        assert (lse.double() - rl).abs().max().item() <= foxtest.TOL_LSE_BF16
        assert lens[now].tolist() == [x[0].shape[0] for x in said]


def test_step_and_copy_in_a_graph(fox):
    """In place, captured once, replayed on new lengths: 20 tokens of every sequence, one at a time."""
    import pagestest

    x = Pool(random.Random(11), 6, 16, 6, 80, 0, idle=0, full=0.3, share=0.8)
    now = x.pages(fox)
    cache = fox.new_cache4(80, 16, 4, 2, 64)
    add, copies = ints([1] * 6), ints([0] * 12, 6, 2)
    ws = fox.pages_workspace(now)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        fox.fox_pages_step(now, add, copies, ws=ws, stream=side)
        fox.fox_cache_copy(cache, copies, ws=ws, stream=side)
    refs, lens, table = list(x.refs), list(x.lens), [list(r) for r in x.table]
    for _ in range(20):
        graph.replay()
        refs, lens, rows, want, short = pagestest.step(refs, lens, table, range(6), [1] * 6, 16, 0, 6)
        table = table_of(rows, 6, 6, table)
        torch.cuda.synchronize()
        assert not short and fox.fox_check_error(ws) == 0
        assert now.refs.tolist() == refs and now.lens.tolist() == lens and now.table.tolist() == table
        assert [tuple(c) for c in copies.tolist()] == want


def test_nothing_to_do(fox):
    """No sequences, no moves, no pairs; a batch that begins from none."""
    refs = ints([0] * 20)
    none = fox.make_pages(16, refs, ints([]), ints([], 0, 5))
    ws = fox.pages_workspace(none)
    fox.fox_pages_step(none, ints([]), ints([], 0, 2), ws=ws)
    mp, used = ints([7] * 20), ints([7, 7])
    fox.fox_pages_compact(none, mp, ints([], 0, 2), used, ws=ws)
    fox.fox_cache_copy(fox.new_cache4(4, 16, 4, 2, 64), ints([], 0, 2))
    assert fox.fox_check_error(ws) == 0 and mp.tolist() == list(range(20)) and used.tolist() == [0, 0]
    two = fox.make_pages(16, ints([-1] * 20), ints([-1, -1]), ints([-1] * 10, 2, 5))
    copies = ints([7] * 4, 2, 2)
    fox.fox_pages_step(none, ints([17, 1]), copies, parent=ints([-1, -1]), out=two)
    assert two.refs.tolist() == [1] * 3 + [0] * 17 and two.lens.tolist() == [17, 1] and copies.tolist() == [[-1, -1]] * 2
    assert two.table.tolist() == [[0, 1, -1, -1, -1], [2, -1, -1, -1, -1]]
    fox.fox_pages_step(two, ints([]), ints([], 0, 2), parent=ints([]), out=none, ws=ws)  # all end
    assert fox.fox_check_error(ws) == 0 and refs.tolist() == [0] * 20


def test_binding_refusals(fox):
    x = Pool(random.Random(1), 4, 16, 4, 60, 0)
    now, out = x.pages(fox), x.blank(fox, 4)
    add, copies = ints([1] * 4), ints([0] * 8, 4, 2)
    with pytest.raises(ValueError):
        fox.fox_pages_step(now, add[:3], copies, out=out)
    with pytest.raises(ValueError):
        fox.fox_pages_step(now, add.long(), copies, out=out)
    with pytest.raises(ValueError):
        fox.fox_pages_step(now, add, copies, parent=add.cpu(), out=out)
    with pytest.raises(fox.FoxError):
        fox.fox_pages_step(now, add, copies, parent=add)  # not in place
    with pytest.raises(fox.FoxError):
        fox.fox_pages_step(now, add, copies, out=fox.make_pages(16, out.refs, out.lens, now.table), parent=add)
    with pytest.raises(fox.FoxError):
        fox.fox_pages_step(now, ints([1] * 5), ints([0] * 10, 5, 2), out=x.blank(fox, 5))
    with pytest.raises(fox.FoxError):
        fox.fox_pages_step(now, add, copies, out=out, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fox.fox_pages_compact(now, ints([0] * 59), ints([0, 0], 1, 2), ints([0, 0]))
    with pytest.raises(ValueError):
        fox.fox_pages_compact(now, ints([0] * 60), ints([0, 0]), ints([0, 0]))
    with pytest.raises(ValueError):
        fox.make_pages(16, now.refs, now.lens, now.table.t())
    cache = fox.new_cache4(4, 16, 4, 2, 64)
    with pytest.raises(ValueError):
        fox.fox_cache_copy(cache, ints([0, 1]))
    with pytest.raises(ValueError):
        fox.fox_cache_copy(cache, ints([[0, 1]]).long())
