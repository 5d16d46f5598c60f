"""Calls that are the first that their host thread makes of CUDA at all: with every output and workspace passed, nothing
before them makes a context current. The same results as on the thread that made the inputs."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def on_a_new_thread(call):
    out = []

    def work():
        try:
            call()
        except Exception as e:
            out.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not out, out


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.fixture(scope="module")
def fox():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    return fox


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 8000])
def test_paged_cache(fox, dtype, prefix):
    from cachetest import Case

    c = Case([50] * 40, [1] * 40, 8, 2, 64, 16, dtype=dtype, uniform=True, prefix=prefix, seed=3)
    c.put()
    cache, batch, s = c.cache(fox), c.batch(fox), torch.cuda.current_stream()
    want = fox.fox_decode(cache, batch, c.q)
    o, lse, ws = torch.empty_like(c.q), torch.empty(40, 8, device="cuda"), fox.cache_workspace(cache, batch, 40)
    k, v, z = c.new_rows()
    on_a_new_thread(lambda: fox.fox_decode(cache, batch, c.q, o=o, lse=lse, ws=ws, stream=s))
    assert torch.equal(bits(o), bits(want[0])) and torch.equal(bits(lse), bits(want[1]))
    on_a_new_thread(lambda: fox.fox_cache_append(cache, batch, k, v, z, ws=ws, stream=s))
    assert fox.fox_check_error(ws) == 0


def test_forward_and_backward(fox):
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v, do = (torch.randn(1, 200, 2, 64, generator=gen, device="cuda").bfloat16() for _ in range(4))
    z = torch.randn(1, 200, 2, generator=gen, device="cuda") + 2
    o, lse = fox.fox_fwd(q, k, v, z)
    want = fox.fox_bwd(q, k, v, z, o, lse, do)
    o2, lse2, grads = torch.empty_like(o), torch.empty_like(lse), [torch.empty_like(t) for t in want]
    ws = fox.workspace(fox.fox_bwd_workspace_bytes(fox.make_params(1, 200, 2, 64)), "cuda")
    s = torch.cuda.current_stream()
    on_a_new_thread(lambda: fox.fox_fwd(q, k, v, z, o=o2, lse=lse2, ws=ws, stream=s))
    assert torch.equal(bits(o2), bits(o)) and torch.equal(bits(lse2), bits(lse))
    names = dict(zip(("dq", "dk", "dv", "dz"), grads))
    on_a_new_thread(lambda: fox.fox_bwd(q, k, v, z, o, lse, do, ws=ws, stream=s, **names))
    assert torch.equal(bits(grads[1]), bits(want[1])) and torch.equal(bits(grads[2]), bits(want[2]))
    assert fox.fox_check_error(ws) == 0
