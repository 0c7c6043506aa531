"""The product's sums where they are hardest: operands whose columns differ
widely in size, sums that cancel, and matrices at any address."""
import pytest
import torch

from tests import layer_common as lc

pytestmark = pytest.mark.gpu


def largest_of_eight(a, b):
    """For each result, the sum over the groups of 8 neighbouring k of the largest
    |a b| of the group."""
    K = a.shape[1]
    out = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for k in range(0, K, 8):
        x, y = a[:, k:k + 8].abs(), b[:, k:k + 8].abs()
        out += (x[:, None] * y[None]).amax(2)
    return out


@pytest.mark.parametrize("M,N,K", [(3, 40, 512), (16, 100, 1000), (32, 70, 640), (64, 130, 1024),
                                   (200, 96, 900), (330, 300, 768)])
@pytest.mark.parametrize("cancel", [False, True])
def test_columns_of_all_sizes(M, N, K, cancel):
    """Columns from 1 to e^6 times as large (outliers), and with `cancel` each large
    column beside its negative.  An fp32 output is an fp32 sum of exact products; for
    a bf16 one each product loses less than 2^-13 of the largest of its group of 8,
    and the sums keep 22 bits."""
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(M + K)
    size = torch.exp(6 * torch.rand(K, generator=g) ** 4)
    x, w = torch.randn(M, K, generator=g) * size, torch.randn(N, K, generator=g)
    if cancel:
        at = torch.arange(0, K - 1, 8)
        x[:, at + 1], w[:, at + 1] = -x[:, at], w[:, at]
    (a, sa), (b, sb) = lc.quantize(x), lc.quantize(w, 128)
    aw, bw = lc.widen(a, sa).cuda(), lc.widen(b, sb, 128).cuda()
    want, total = aw @ bw.t(), aw.abs() @ bw.abs().t()
    args = [t.cuda() for t in (a, sa.view(lc.E8), b, sb.view(lc.E8))]
    lc.bound(m.fp8_matmul(*args, out_dtype=torch.float32), want, (K + 4) * lc.U32 * total, torch.float32)
    lc.bound(m.fp8_matmul(*args), want, 8 * 2.0 ** -13 * largest_of_eight(aw, bw)
             + (K / 8 + 4) * 2.0 ** -22 * total, torch.bfloat16)


@pytest.mark.parametrize("M,N", [(16, 64), (64, 64), (300, 300), (2048, 4096)])
def test_beside_a_pair_that_cancels(M, N):
    """P - P + p in one group of 8: p to fp32 sums' precision in fp32, within 2^-13 of
    P in bf16; in another group whole in bf16."""
    import selective_state_space_52_amd as m
    K, P = 128, 2.0 ** 16
    one = torch.full((M, 1), 127, dtype=torch.uint8).view(lc.E8).cuda()
    two = torch.full((N, 1), 127, dtype=torch.uint8).view(lc.E8).cuda()
    for at in (2, 7, 8, 127):
        a, b = torch.zeros(M, K), torch.zeros(N, K)
        a[:, 0], a[:, 1], b[:, :2], a[:, at] = 256, -256, 256, 1.75
        b[:, at] = torch.tensor([2.0 ** (n % 14 - 5) for n in range(N)])
        want = (a.double() @ b.double().t())
        args = (a.to(lc.F8).cuda(), one, b.to(lc.F8).cuda(), two)
        err = (m.fp8_matmul(*args, out_dtype=torch.float32).cpu().double() - want).abs()
        assert float(err.max()) <= 3 * lc.U32 * 2 * P      # three terms
        err = (m.fp8_matmul(*args).cpu().double() - want).abs()
        assert float(err.max()) < (2.0 ** -13 * P if at < 8 else 2.0 ** -30)


@pytest.mark.parametrize("M,N,K", [(9, 70, 256), (30, 40, 528), (100, 130, 320), (400, 300, 388),
                                   (700, 700, 512), (2900, 4500, 144)])
def test_any_address(M, N, K):
    """Operands, scales and results that start 1 to 12 bytes (results: elements)
    past an aligned address: the same bits as the aligned ones'."""
    import selective_state_space_52_amd as m
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, generator=g, device="cuda")
    w = torch.randn(N, K, generator=g, device="cuda")
    ops = [*m.quantize_fp8(x), *m.quantize_fp8(w, block_rows=128)]

    def moved(t, by):
        flat = torch.zeros(t.numel() + 16, dtype=torch.uint8, device="cuda")
        out = flat[by:by + t.numel()].view(t.shape)
        out.copy_(t.view(torch.uint8))
        return out.view(t.dtype)
    for dtype in (torch.bfloat16, torch.float32):
        want = m.fp8_matmul(*ops, out_dtype=dtype)
        for by in ((1, 0, 0, 0), (0, 0, 2, 0), (4, 0, 0, 0), (0, 0, 8, 0), (12, 1, 4, 3), (8, 2, 8, 1), (3, 3, 5, 2)):
            at = [moved(t, n) for t, n in zip(ops, by)]
            assert [t.data_ptr() % 16 for t in at] == list(by)
            assert torch.equal(m.fp8_matmul(*at, out_dtype=dtype), want), by
        for by in (1, 2, 3):
            flat = torch.full((M * N + 8,), 7.0, dtype=dtype, device="cuda")
            got = m.fp8_matmul(*ops, out=flat[by:by + M * N].view(M, N))
            assert torch.equal(got, want)
            assert bool((flat[:by] == 7).all()) and bool((flat[by + M * N:] == 7).all())
