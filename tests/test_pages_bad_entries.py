"""Table entries that are no pages of the pool, in sequences that go on: reported by the step, and nothing else is touched by them."""
import random

import pytest

from test_pages_parity import FOX_ERR_DEVICE, MARK, Pool, ints, table_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    fox.lib()
    return fox


@pytest.mark.parametrize("bad", [100, -1, 2**31 - 1, -(2**31)])
@pytest.mark.parametrize("stride", [8, 700])  # references counted by the step itself, and by a kernel of their own
@pytest.mark.parametrize("how,entry", [("one child", 2), ("one child", 1), ("two children", 0), ("ends", 2), ("apart", 2), ("apart", 1),
                                       ("in place", 2), ("in place", 1)])
def test_entries_outside_the_pool(fox, how, entry, stride, bad):
    import pagestest

    B = 6
    x = Pool(random.Random(5), B, 16, stride, 100, 40, idle=0, share=0, full=3 / stride)  # all of them fit
    x.lens[2] = x.P + 37  # two pages and a part
    free = [i for i in range(100) if x.refs[i] == 0]
    for c in range(3):
        if x.table[2][c] == MARK:
            x.table[2][c] = free.pop()
    x.refs = [0] * 100
    for i in x.prefix_table:
        x.refs[i] += 1
    for b in range(B):
        for c in range(pagestest.pages_of(x.lens[b] - x.P, 16)):
            x.refs[x.table[b][c]] += 1
    x.refs[x.table[2][entry]] -= 1
    x.table[2][entry] = bad
    parent = list(range(B))
    if how == "two children":
        parent[4] = 2
    elif how == "ends":
        parent[2] = -1
    add = [3, 0, 5, 1, 40, 2]
    # the definition, with the entry a page behind the pool that is held once and is never free
    model = [list(r) for r in x.table]
    model[2][entry] = 100
    refs, lens, rows, copies, short = pagestest.step(x.refs + [1 if how != "ends" else 2], x.lens, model, parent, add, 16, x.P, B)
    assert not short
    now = x.pages(fox)
    out = now if how == "in place" else x.blank(fox, B)
    got = torch.full((B, 2), MARK, dtype=torch.int32, device="cuda")
    ws = fox.pages_workspace(now, out)
    fox.fox_pages_step(now, ints(add), got, parent=None if how in ("apart", "in place") else ints(parent),
                       out=None if how == "in place" else out, ws=ws)
    # in place only a last page that is grown into is looked at
    assert fox.fox_check_error(ws) == (0 if (how, entry) == ("in place", 1) else FOX_ERR_DEVICE)
    assert fox.fox_check_error(ws) == 0
    assert out.refs.tolist() == refs[:100]
    assert out.lens.tolist() == lens
    want = table_of(rows, B, stride, model if how == "in place" else None)
    assert out.table.tolist() == [[bad if e == 100 else e for e in r] for r in want]
    assert [tuple(c) for c in got.tolist()] == copies
