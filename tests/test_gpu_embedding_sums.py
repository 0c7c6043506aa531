"""The embedding's gradient where its sums are exact, so that a row lost, doubled or
put to another token shows in every bit."""
import pytest
import torch

from tests import layer_common as lc
from tests.test_gpu_embedding import KINDS, tokens_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,dim", [(300, 41, 20), (513, 5000, 9), (1777, 50257, 24), (5000, 300, 520),
                                            (8192, 50304, 16), (70001, 3001, 24), (70001, 130000, 8)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("io,add", [("f32", False), ("bf16", True)])
def test_whole_numbers(rows, vocab, dim, kind, io, add):
    """Whole numbers up to 8: sums below 2^24, exact in fp32 in any order."""
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(rows + vocab)
    t = tokens_of(kind, rows, vocab, g)
    dout = torch.randint(-8, 9, (rows, dim), generator=g)
    old = torch.randint(-99, 100, (vocab, dim), generator=g) if add else None
    got = m.embedding_bwd(t.cuda(), dout.to(lc.IO[io]).cuda(), vocab,
                          add_to=None if old is None else old.float().cuda())
    live = (t >= 0) & (t < vocab)
    want = torch.zeros(vocab, dim, dtype=torch.int64) if old is None else old.clone()
    want.index_add_(0, t[live], dout[live])
    assert torch.equal(got.cpu(), want.float())
