"""Top-k on both sides of the longest list that is ranked pair by pair (256
tokens) and of a workgroup's threads (1024)."""
import pytest
import torch

from tests.test_gpu_sample import check, random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top_k", [180, 255, 256, 257, 300, 1023, 1024, 1025])
@pytest.mark.parametrize("vocab", [257, 4099, 50304])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_k(top_k, vocab, dtype):
    logits, noise = random(4, vocab, top_k, dtype=dtype)
    check(logits, noise, top_k=top_k)
    check(logits, noise, top_k=top_k, top_p=0.9, min_p=0.001, per_row=False)


def test_no_pass_for_nothing():
    """A top-k that no list can hold takes the same path on either side of the
    number of threads, so it takes the same time."""
    import selective_state_space_52_amd as m
    logits, noise = random(256, 50304, 1, dtype=torch.bfloat16)
    logits, noise = logits.cuda(), noise.cuda()

    def graph(k):
        m.sample_tokens(logits, noise, top_k=k)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                m.sample_tokens(logits, noise, top_k=k)
        return g
    graphs, best = {k: graph(k) for k in (1024, 1025)}, {1024: 1e9, 1025: 1e9}
    for _ in range(20):
        for k, g in graphs.items():
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            g.replay()
            end.record()
            end.synchronize()
            best[k] = min(best[k], start.elapsed_time(end))
    assert best[1024] < 1.12 * best[1025]
