"""The embedding's rows and their gradient against 64-bit references."""
import pytest
import torch

from tests import layer_common as lc
from tests import train_common as tc

pytestmark = pytest.mark.gpu


def tokens_of(kind, rows, vocab, g):
    if kind == "same":
        return torch.full((rows,), vocab // 2)
    t = torch.randint(0, vocab, (rows,), generator=g)
    if kind == "skewed":      # most rows have a few tokens
        few = torch.randint(0, vocab, (3,), generator=g)
        t = torch.where(torch.rand(rows, generator=g) < 0.8, few[torch.randint(0, 3, (rows,), generator=g)], t)
    elif kind == "ordered":   # a vocabulary in order of frequency
        t = (vocab ** torch.rand(rows, generator=g, dtype=torch.float64)).long() - 1
    elif kind == "padded":
        out = torch.tensor([-1, vocab, -(1 << 40), 1 << 40, (1 << 32) + 1, -(1 << 63)])
        t = torch.where(torch.rand(rows, generator=g) < 0.5,
                        out[torch.randint(0, len(out), (rows,), generator=g)], t)
    elif kind == "none":
        t = torch.full((rows,), -1)
    return t


@pytest.mark.parametrize("rows,vocab,dim", [(1, 1, 1), (3, 5, 7), (2, 300, 8), (65, 33, 100), (7, 11, 512),
                                            (130, 1000, 513), (5, 17, 2560), (2, 3, 9001)])
@pytest.mark.parametrize("table,io", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("scale", [1.0, 22.6])
def test_forward(rows, vocab, dim, table, io, scale):
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(rows + dim)
    w = torch.randn(vocab, dim, generator=g).to(lc.IO[table])
    t = tokens_of("padded" if rows > 2 else "even", rows, vocab, g)
    out = m.embedding_fwd(t.cuda(), w.cuda(), scale=scale, out_dtype=lc.IO[io])
    want = tc.embedding(t, w, scale)
    # the scale is fp32 too
    lc.bound(out, want, 0.0 if scale == 1 else 2 * lc.U32 * want.abs(), lc.IO[io])
    if scale == 1:
        same = m.embedding_fwd(t.cuda(), w.cuda())
        assert same.dtype == w.dtype and torch.equal(same.cpu(), tc.embedding(t, w, 1.0).to(w.dtype))


KINDS = ["even", "same", "skewed", "ordered", "padded", "none"]


@pytest.mark.parametrize("rows,vocab,dim", [(1, 1, 1), (1, 50, 64), (31, 7, 9), (32, 300, 33), (33, 2, 512),
                                            (64, 1000, 520), (257, 257, 130), (1500, 515, 70),
                                            (2100, 40, 1030), (1030, 5000, 8), (1024, 90, 40),
                                            (1025, 90, 1040), (100, 9001, 3), (1100, 9001, 1),
                                            (512, 90, 40), (513, 90, 600)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("io,grad,add", [("bf16", "f32", False), ("f32", "f32", True),
                                         ("bf16", "bf16", True), ("f32", "bf16", False)])
def test_backward(rows, vocab, dim, kind, io, grad, add):
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(rows * 3 + dim)
    t = tokens_of(kind, rows, vocab, g)
    dout = torch.randn(rows, dim, generator=g).to(lc.IO[io])
    dout[(t < 0) | (t >= vocab)] = float("nan")        # padding's are not read
    old = torch.randn(vocab, dim, generator=g).to(lc.IO[grad]) if add else None
    td, dd = t.cuda(), dout.cuda()

    def call():
        if add:
            return m.embedding_bwd(td, dd, vocab, scale=0.7, add_to=old.cuda())
        return m.embedding_bwd(td, dd, vocab, scale=0.7, out_dtype=lc.IO[grad])
    got, again = call(), call()
    assert torch.equal(got, again)
    want, size = tc.embedding_bwd(t, dout, vocab, 0.7)
    slack = lc.U32 * (size + 3 * want.abs())
    if add:
        named = torch.zeros(vocab, dtype=torch.bool)
        named[t[(t >= 0) & (t < vocab)]] = True
        assert torch.equal(got.cpu()[~named], old[~named])
        want = want + old.double()
        slack = slack + lc.U32 * want.abs()
    lc.bound(got, want, slack, lc.IO[grad])


@pytest.mark.parametrize("kind", ["even", "same", "skewed", "ordered"])
def test_backward_long(kind):
    """Many pieces of the order, tokens across hundreds of them."""
    import selective_state_space_52_amd as m
    rows, vocab, dim = 70001, 3001, 24
    g = torch.Generator().manual_seed(5)
    t = tokens_of(kind, rows, vocab, g)
    dout = torch.randn(rows, dim, generator=g)
    got = m.embedding_bwd(t.cuda(), dout.cuda(), vocab)
    want = torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, t, dout.double())
    size = torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, t, dout.double().abs())
    count = torch.bincount(t, minlength=vocab)
    lc.bound(got, want, lc.U32 * size * (count[:, None] + 4), torch.float32)


def test_tables_past_32_bits():
    """Rows whose elements lie beyond 2^31, and a vocabulary of 2^20 and more."""
    import selective_state_space_52_amd as m
    vocab, dim = (1 << 20) + 5, 2100
    t = torch.tensor([vocab - 1, 0, 1 << 20, vocab - 1, 7], device="cuda")
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table[t] = torch.randn(5, dim, device="cuda").bfloat16()
    assert torch.equal(m.embedding_fwd(t, table), table[t])
    dout = torch.randn(5, dim, device="cuda").bfloat16()
    got = m.embedding_bwd(t, dout, vocab, out_dtype=torch.bfloat16)
    want = (dout[0].float() + dout[3].float()).bfloat16()
    assert torch.equal(got[vocab - 1], want) and torch.equal(got[t[1:3]], dout[1:3])
    got[t] = 0
    assert not got.view(torch.int16).any()


@pytest.mark.parametrize("add", [False, True])
def test_sorted_rows_of_a_long_table(add):
    """More rows than are compared directly, into a table of more rows than 256
    workgroups order."""
    import selective_state_space_52_amd as m
    rows, vocab, dim = 2500, (1 << 20) + 5, 9
    g = torch.Generator().manual_seed(4)
    t = torch.randint(0, vocab, (rows,), generator=g)
    t[::3] = torch.randint(vocab - 40, vocab, (len(t[::3]),), generator=g)
    t[0], t[1] = 0, -1
    dout = torch.randn(rows, dim, generator=g)
    old = torch.randn(vocab, dim, generator=g)
    got = m.embedding_bwd(t.cuda(), dout.cuda(), vocab, add_to=old.cuda() if add else None)
    live = t >= 0
    want = torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, t[live], dout[live].double())
    size = torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, t[live], dout[live].double().abs())
    count = torch.bincount(t[live], minlength=vocab)[:, None]
    slack = lc.U32 * size * (count + 4)
    if add:
        want = want + old.double()
        slack = slack + lc.U32 * want.abs() * (count > 0)
    lc.bound(got, want, slack, torch.float32)


def test_strided_rows_and_other_streams():
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(1)
    t = torch.randint(0, 99, (200,), generator=g).cuda()
    wide = torch.randn(200, 300, generator=g).bfloat16().cuda()
    view = wide[:, 3:250]
    got = m.embedding_bwd(t, view, 99)
    assert torch.equal(got, m.embedding_bwd(t, view.contiguous(), 99))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = m.embedding_bwd(t, view, 99)
    side.synchronize()
    assert torch.equal(got, other)
    # a captured call, replayed with new tokens and eager work in between
    tokens, dout = t.clone(), view.contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.embedding_bwd(tokens, dout, 99)
        rows = m.embedding_fwd(tokens, out)
    for k in range(4):
        tokens.copy_(torch.randint(0, 99, (200,), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = m.embedding_bwd(tokens, dout, 99)
        assert torch.equal(out, want) and torch.equal(rows, want[tokens])


def test_gradient_against_differences():
    """The lookup is linear in the table: differences along random directions are
    exact but for their own rounding."""
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(2)
    t = tokens_of("padded", 60, 20, g)
    dout = torch.randn(60, 40, generator=g)
    got = m.embedding_bwd(t.cuda(), dout.cuda(), 20, scale=3.0).cpu().double()
    for _ in range(3):
        way = torch.randn(20, 40, generator=g, dtype=torch.float64)
        diff = float((tc.embedding(t, way, 3.0) * dout.double()).sum())
        assert abs(diff - float((got * way).sum())) <= 70 * lc.U32 * float((got * way).abs().sum()) + \
            70 * lc.U32 * float((tc.embedding(t, way, 3.0) * dout.double()).abs().sum())


def test_refusals():
    import selective_state_space_52_amd as m
    t, w = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(9, 16, device="cuda")
    d = torch.zeros(4, 16, device="cuda")
    for call in (lambda: m.embedding_fwd(t.int(), w), lambda: m.embedding_fwd(t[None], w),
                 lambda: m.embedding_fwd(t, w.half()), lambda: m.embedding_fwd(t, w.t()),
                 lambda: m.embedding_fwd(t.cpu(), w), lambda: m.embedding_fwd(t, w, out_dtype=torch.half),
                 lambda: m.embedding_bwd(t[:3], d, 9), lambda: m.embedding_bwd(t, d.t(), 9),
                 lambda: m.embedding_bwd(t, d, 9, add_to=w[:8]),
                 lambda: m.embedding_bwd(t, d, 9, add_to=w.half())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.MssmError):
        m.embedding_fwd(t[:0], w)
    with pytest.raises(m.MssmError):
        m.embedding_bwd(t, d, 0)
