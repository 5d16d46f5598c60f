"""Gate projections from several host threads at once, with different head counts: a kernel's limit of shared memory
belongs to the function, so that a call with few heads must not lower it between another's setting and launch."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_host_threads_with_different_head_counts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import forget_gated_softmax_gb300 as fox

    jobs = []
    for H in (4, 256, 40):
        gen = torch.Generator("cuda").manual_seed(H)
        x = torch.randn(1, 100, 64, generator=gen, device="cuda").bfloat16()
        w = torch.randn(H, 64, generator=gen, device="cuda").bfloat16()
        b = torch.randn(H, generator=gen, device="cuda")
        ws = fox.workspace(fox.fox_fwd_workspace_bytes(fox.make_params(1, 100, H, 64)), "cuda")
        z = torch.empty(1, 100, H, device="cuda")
        jobs.append((x, w, b, ws, z, torch.cuda.Stream(), fox.fox_gate_proj(x, w, b)))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        x, w, b, ws, z, stream, _ = job
        try:
            torch.cuda.set_device(0)
            for _ in range(6000):
                fox.fox_gate_proj(x, w, b, z=z, ws=ws, stream=stream)
        except Exception as e:
            failed.append((w.shape[0], e))

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for *_, ws, z, _, want in jobs:
        assert torch.equal(z, want)
        assert fox.fox_check_error(ws) == 0
