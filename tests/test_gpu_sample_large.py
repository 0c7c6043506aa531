"""Sampling from large vocabularies without ties, whose boundary bin holds more
tokens than the list in LDS: the boundary is found digit by digit."""
import pytest
import torch

from tests.test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [100003, 128256, 256000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", [dict(top_p=0.95), dict(top_p=0.99), dict(top_p=0.95, temperature=1.3),
                                      dict(top_k=30000), dict(top_k=90000, top_p=0.97, min_p=1e-6)])
def test_wide_bins(vocab, dtype, settings):
    g = torch.Generator().manual_seed(vocab)
    logits = 2.5 * torch.randn(3, vocab, generator=g)
    hot = torch.randint(0, vocab, (3, 20), generator=g)
    logits.scatter_add_(1, hot, 4 + 4 * torch.rand(3, 20, generator=g))
    check(logits.to(dtype), torch.rand(3, vocab, generator=g), **settings)
