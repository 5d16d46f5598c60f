"""Decode calls from several host threads at once, each with a stream, a workspace and outputs of its own.

A kernel's limit of shared memory belongs to the function, not to a call: a thread with a small batch must not
lower it between another's setting and launch. Every status is FOX_OK, and the results are those of a call alone."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CALLS = 6000

# one kernel each; batches whose calls take different amounts of shared memory: own, heads, key heads, d, page, prefix
PAIRS = {
    "f32": ("f32", [([5], 8, 2, 64, 16, 0), ([5] * 2048, 8, 2, 64, 16, 0), ([9] * 40, 8, 2, 64, 16, 0)]),
    "bf16": ("bf16", [([5], 8, 2, 128, 64, 0), ([5] * 2048, 8, 2, 128, 64, 0), ([9] * 40, 8, 2, 128, 16, 0)]),
    "prefix": ("bf16", [([5] * 129, 1, 1, 64, 64, 4000), ([5] * 9, 20, 1, 64, 64, 20000), ([5] * 40, 4, 1, 64, 64, 8000)]),
}


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("which", list(PAIRS))
def test_host_threads_with_batches_of_different_sizes(which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox
    from cachetest import Case

    dtype, shapes = PAIRS[which]
    jobs = []
    for n, (own, H, Hkv, d, S, P) in enumerate(shapes):
        c = Case(own, [1] * len(own), H, Hkv, d, S, dtype=dtype, uniform=True, prefix=P, seed=60 + n)
        c.put()
        cache, batch = c.cache(fox), c.batch(fox)
        o, lse = torch.empty_like(c.q), torch.empty(len(own), H, device="cuda")
        jobs.append((c, cache, batch, fox.cache_workspace(cache, batch, len(own)), o, lse, torch.cuda.Stream(),
                     fox.fox_decode(cache, batch, c.q)))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        c, cache, batch, ws, o, lse, stream, _ = job
        try:
            torch.cuda.set_device(0)
            for _ in range(CALLS):
                fox.fox_decode(cache, batch, c.q, o=o, lse=lse, ws=ws, stream=stream)
        except Exception as e:
            failed.append((len(c.own), e))

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for _, _, _, ws, o, lse, _, want in jobs:
        assert torch.equal(bits(o), bits(want[0])) and torch.equal(bits(lse), bits(want[1]))
        assert fox.fox_check_error(ws) == 0
