"""The layer's operators over arrays of more than 2^31 elements, checked on
rows on both sides of element 2^31 against the same rows alone or in 64 bits."""
import pytest
import torch

from tests import layer_common as lc

pytestmark = pytest.mark.gpu
EDGE = 2 ** 31


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def fill(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(generator=g)


def test_norm():
    import selective_state_space_52_amd as m
    dim = 2560
    rows = EDGE // dim + 3000
    x, w = fill(rows, dim, dtype=torch.bfloat16, seed=1), fill(dim, dtype=torch.float32, seed=2)
    q, scales, _, rstd = m.rms_norm_fwd_fp8(x, w, want_rstd=True)
    for a in (0, EDGE // dim - 2, rows - 4):
        at = slice(a, a + 4)
        q2, s2, _, r2 = m.rms_norm_fwd_fp8(x[at], w, want_rstd=True)
        assert torch.equal(q[at].view(torch.uint8), q2.view(torch.uint8))
        assert torch.equal(scales[at].view(torch.uint8), s2.view(torch.uint8))
        assert torch.equal(rstd[at], r2)
    del q
    dout = fill(rows, dim, dtype=torch.bfloat16, seed=3)
    dx, _, dw = m.rms_norm_bwd(dout, x, w, rstd)
    for a in (0, EDGE // dim - 2, rows - 4):
        at = slice(a, a + 4)
        one, _, _ = m.rms_norm_bwd(dout[at], x[at], w, rstd[at])
        assert torch.equal(dx[at], one)
    want, size = torch.zeros(dim, dtype=torch.float64, device="cuda"), 0
    for a in range(0, rows, 1 << 16):
        at = slice(a, a + (1 << 16))
        t = dout[at].float() * (x[at].float() * rstd[at, None])
        want += t.sum(0, dtype=torch.float64)
        size = size + t.abs().sum(0, dtype=torch.float64)
    # fp32 sums over this many rows by 3 rounds of partial sums: each adds at most
    # one rounding of its running sum a term
    blocks = 3 * 256
    lc.bound(dw, want, (rows / blocks + blocks + 8) * lc.U32 * size, torch.float32)


def test_quantize_and_product():
    import selective_state_space_52_amd as m
    rows, cols = 46400, 46400
    x = fill(rows, cols, dtype=torch.bfloat16, seed=4)
    q, s = m.quantize_fp8(x, transpose=True)
    edge = EDGE // rows     # the row of q that holds element 2^31
    for a in (0, edge, cols - 128):
        q2, s2 = m.quantize_fp8(x[:, a:a + 128], transpose=True)
        assert torch.equal(q[a:a + 128].view(torch.uint8), q2.view(torch.uint8))
        assert torch.equal(s[a:a + 128].view(torch.uint8), s2.view(torch.uint8))
    del x
    # operands of more than 2^31 values
    b, bs = m.quantize_fp8(fill(16, rows, dtype=torch.bfloat16, seed=5))
    for dtype in (torch.bfloat16, torch.float32):
        out = m.fp8_matmul(q, s, b, bs, out_dtype=dtype)
        for a in (0, edge // 192 * 192, cols - 200):
            one = lc.widen(q[a:a + 200].cpu(), s[a:a + 200].view(torch.uint8).cpu())
            two = lc.widen(b.cpu(), bs.view(torch.uint8).cpu())
            want = one @ two.t()
            slack = (rows + 4) * lc.U32 * (one.abs() @ two.abs().t())
            if dtype == torch.bfloat16:   # products to 2^-17 of their block's largest
                slack = slack + 8 * 2.0 ** -17 * rows ** 0.5 * one.abs().amax(1)[:, None] * two.abs().amax(1)
            lc.bound(out[a:a + 200], want, slack, dtype)


def test_product_output():
    import selective_state_space_52_amd as m
    M, N, K = 46400, 46400, 128
    a, sa = m.quantize_fp8(fill(M, K, dtype=torch.bfloat16, seed=6))
    b, sb = m.quantize_fp8(fill(N, K, dtype=torch.bfloat16, seed=7), block_rows=128)
    out = m.fp8_matmul(a, sa, b, sb)
    wide = lc.widen(b, sb.view(torch.uint8), 128)
    for r in (0, EDGE // N, M - 1):
        want = lc.widen(a[r:r + 1], sa[r:r + 1].view(torch.uint8)) @ wide.t()
        assert float((out[r].double() - want[0]).norm() / want.norm()) < 2 * lc.U16


def test_sample():
    import selective_state_space_52_amd as m
    vocab = 65600
    rows = EDGE // vocab + 40
    logits = fill(rows, vocab, dtype=torch.bfloat16, seed=8)
    noise = torch.empty(rows, vocab, device="cuda").uniform_(generator=torch.Generator("cuda").manual_seed(9))
    tokens, lp = m.sample_tokens(logits, noise, top_p=0.9, min_p=0.01)
    for a in (0, EDGE // vocab - 2, rows - 4):
        t2, l2 = m.sample_tokens(logits[a:a + 4], noise[a:a + 4], top_p=0.9, min_p=0.01)
        assert torch.equal(tokens[a:a + 4], t2) and torch.equal(lp[a:a + 4], l2)


def test_step_in_a_long_cache():
    import selective_state_space_52_amd as m
    heads, N = 80, 128
    dim, ch = heads * 64, heads * 64 + 2 * N
    cache = EDGE // (dim * N) + 40
    g = torch.Generator(device="cuda").manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state = fill(cache, dim, N, dtype=torch.float32, seed=11)
    window = fill(cache, ch, 3, dtype=torch.bfloat16, seed=12)
    edge = EDGE // (dim * N)
    at = torch.tensor([0, edge - 1, edge, cache - 1], device="cuda")
    args = dict(conv_weight=r(ch, 4), A=-r(heads).abs(), conv_bias=r(ch), D=r(heads), dt_bias=r(heads) - 3)
    xbc, dt, z = r(4, ch).bfloat16(), r(4, heads).bfloat16(), r(4, dim).bfloat16()
    few, few_window = state[at].contiguous(), window[at].contiguous()
    before = state[1].clone()
    out = m.mamba2_state_update(state, window, xbc, dt, z=z, slots=at.int(), **args)
    want = m.mamba2_state_update(few, few_window, xbc, dt, z=z, **args)
    assert torch.equal(out, want) and torch.equal(state[at], few) and torch.equal(window[at], few_window)
    assert torch.equal(state[1], before)
