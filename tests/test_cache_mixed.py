"""Decode of batches whose sequences bring very different counts of new tokens, on the GPU."""
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

    return fox


def Case(*a, **kw):
    from cachetest import Case

    return Case(*a, **kw)


def check(fox, c, dtype, label, bias_from_j=False):
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    ws[fox.FOX_CACHE_ZERO_BYTES :] = 0xFF  # nothing is read that the call has not written
    o, lse = torch.full_like(c.q, float("nan")), torch.full((c.rows, c.H), float("nan"), device="cuda")
    fox.fox_decode(cache, batch, c.q, bias_from_j=bias_from_j, o=o, lse=lse, ws=ws)
    assert fox.fox_check_error(ws) == 0
    last = sum(c.new)
    assert torch.isnan(o[last:]).all() and torch.isnan(lse[last:]).all()
    ro, rl = c.attend(bias_from_j=bias_from_j)
    idle = torch.isinf(rl[:last])
    assert torch.equal(idle, torch.isinf(lse[:last])) and (o[:last][idle] == 0).all()
    assert_o(tensor_f64(o[:last]), tensor_f64(ro[:last]), dtype, label)
    tol = foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32
    assert (lse[:last].double() - rl[:last])[~idle].abs().max().item() <= tol
    again = fox.fox_decode(cache, batch, c.q, bias_from_j=bias_from_j, ws=ws)
    assert torch.equal(again[0][:last], o[:last]) and torch.equal(again[1][:last], lse[:last])


def mixed(B, prompts, seed=0):
    """New tokens of B sequences: mostly one, some none, `prompts` {place: tokens}; own tokens of each, some idle."""
    new = [prompts.get(b, 0 if (b + seed) % 7 == 3 else 1) for b in range(B)]
    own = [None if b % 9 == 5 else x + (b * 37) % 150 for b, x in enumerate(new)]
    return own, new


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,prompts,H,Hkv,d,S,prefix", [
    (30, {11: 300}, 8, 2, 128, 64, 0),
    (30, {0: 200, 29: 130}, 14, 2, 64, 16, 0),
    (40, {39: 257}, 20, 1, 128, 128, 0),
    (12, {3: 500, 4: 33}, 4, 4, 64, 32, 70),
    (300, {150: 100}, 8, 2, 64, 16, 0),
])
def test_prompts_among_single_tokens(fox, dtype, B, prompts, H, Hkv, d, S, prefix):
    own, new = mixed(B, prompts, seed=d)
    c = Case(own, new, H, Hkv, d, S, dtype=dtype, prefix=prefix, seed=B, tail=2)
    c.put()
    check(fox, c, dtype, f"decode mixed {B} {dtype}", bias_from_j=d == 64)


def test_prompts_among_single_tokens_behind_a_shared_prefix(fox):
    own, new = mixed(40, {17: 150}, seed=1)
    c = Case(own, new, 8, 2, 128, 64, prefix=5003, seed=2, tail=1)
    c.put()
    fox.trace_begin()
    check(fox, c, "bf16", "decode mixed shared")
    assert "prefix" in [k for k, _ in fox.trace_end()]


@pytest.mark.parametrize("dtype,prefix", [("bf16", 0), ("f32", 0), ("bf16", 5003)])
def test_rows_that_begin_before_an_earlier_end_are_left_out(fox, dtype, prefix):
    """Row ranges out of order, each of them one that the batch holds: reported, the later sequence left out, the rows
    of the others as they are."""
    new = [60, 1, 1, 1] + [1] * 28
    own = [x + 70 for x in new]
    c = Case(own, new, 8, 2, 128, 64, dtype=dtype, prefix=prefix, seed=3)
    c.put()
    want_o, want_l = c.attend()
    cache, batch = c.cache(fox), c.batch(fox)
    ws = fox.cache_workspace(cache, batch, c.rows)
    cu = c.cu.clone()
    # sequence 1 would begin inside the first one's rows (behind a falling entry), sequence 2 and those behind it as before
    c.cu[1], c.cu[2] = 60, 30
    c.cu[3] = 62
    o, lse = torch.full_like(c.q, float("nan")), torch.full((c.rows, 8), float("nan"), device="cuda")
    fox.fox_decode(cache, batch, c.q, o=o, lse=lse, ws=ws)
    assert fox.fox_check_error(ws) == FOX_ERR_DEVICE
    live = [r for r in range(c.rows) if not 30 <= r < 62]  # all but the rows that the sequence left out claims
    assert torch.isnan(o[60:62]).all() and torch.isnan(lse[60:62]).all()
    assert_o(tensor_f64(o[live]), tensor_f64(want_o[live]), dtype, "decode beside falling rows")
    tol = foxtest.TOL_LSE_BF16 if dtype == "bf16" else foxtest.TOL_LSE_F32
    assert (lse[live].double() - want_l[live]).abs().max().item() <= tol
    c.cu.copy_(cu)
    check(fox, c, dtype, "decode after falling rows")
