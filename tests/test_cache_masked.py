"""Infinities and NaN in what a row does not attend to: the keys, gates and values of new tokens behind its position."""
import pytest

import foxtest
from foxtest import assert_o, tensor_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    return fox


def Case(*a, **kw):
    from cachetest import Case

    return Case(*a, **kw)


# own, new, H, Hkv, d, page, prefix
CASES = [
    ([40, 9], [4, 9], 8, 2, 128, 64, 0),        # a few tokens, one row tile (grouped heads)
    ([33, 64, 100], [2, 3, 7], 4, 4, 64, 16, 0),
    ([70, 300], [70, 130], 8, 2, 128, 32, 0),   # many row tiles: keys seen by all, some and no rows of each
    ([50], [40], 20, 1, 64, 128, 0),            # a group of more heads than a row tile
    ([30, 41], [5, 2], 6, 2, 128, 64, 77),      # behind a walked prefix
    ([25] * 40, [4] * 40, 8, 2, 64, 16, 5003),  # behind a shared one (bf16)
    ([5000, 9], [6, 3], 8, 2, 128, 64, 0),      # split among workers
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", range(len(CASES)))
def test_values_behind_a_row_s_position(fox, n, dtype):
    """V of some new tokens holds infinities and NaN in some channels: rows before them are as if it held zeros, and so
    are the other channels of the rows that see them; those channels are no numbers there."""
    own, new, H, Hkv, d, S, P = CASES[n]
    c = Case(own, new, H, Hkv, d, S, dtype=dtype, prefix=P, seed=30 + n)
    bad, hit = [], torch.zeros(c.rows, Hkv, d, dtype=torch.bool, device="cuda")
    for b in range(c.B):
        first = own[b] - new[b]
        for i, t in enumerate({1, new[b] // 2, new[b] - 1} - {0} if new[b] > 1 else set()):
            for h, ch, v in ((0, (7 * t) % d, INF), (Hkv - 1, (5 * t + 3) % d, NAN), (0, d - 1, -INF)):
                c.seq[b][1][first + t, h, ch] = 0.0
                bad.append((b, first + t, h, ch, v))
                hit[c.row0[b] + t : c.row0[b] + new[b], h, ch] = True
    ro, rl = c.attend()
    for b, t, h, ch, v in bad:
        c.seq[b][1][t, h, ch] = v
    c.put()
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    o, lse = fox.fox_decode(cache, batch, c.q, ws=ws)
    assert fox.fox_check_error(ws) == 0
    hit = hit.repeat_interleave(H // Hkv, 1)
    assert not torch.isfinite(o[hit]).any()
    assert torch.isfinite(o[~hit]).all()
    o, ro = torch.where(hit, 0.0, o.double()), torch.where(hit, 0.0, ro)
    assert_o(tensor_f64(o), tensor_f64(ro), dtype, f"decode masked {n} {dtype}")
    tol = foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32
    assert (lse.double() - rl).abs().max().item() <= tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", range(len(CASES)))
def test_keys_and_gates_behind_a_row_s_position(fox, n, dtype):
    """NaN in K and in the gates' sums of each sequence's last new token: the rows before it do not change."""
    own, new, H, Hkv, d, S, P = CASES[n]
    c = Case(own, new, H, Hkv, d, S, dtype=dtype, prefix=P, seed=50 + n)
    c.put()
    cache, batch = c.cache(fox), c.batch(fox)
    o, lse = fox.fox_decode(cache, batch, c.q)
    last = torch.tensor([c.row0[b] + new[b] - 1 for b in range(c.B)], device="cuda")
    for b in range(c.B):
        page, slot = int(c.table[b, (own[b] - 1) // S]), (own[b] - 1) % S
        c.k[page, :, slot] = NAN if b % 2 else INF
        c.g[page, :, slot] = NAN
    o2, lse2 = fox.fox_decode(cache, batch, c.q)
    keep = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    keep[last] = False
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])
