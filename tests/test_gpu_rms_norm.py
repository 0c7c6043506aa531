"""The norm with the residual's addition, its 8-bit output and its backward,
against 64-bit references."""
import pytest
import torch

from tests import layer_common as lc

pytestmark = pytest.mark.gpu
EPS = 1e-5


def inputs(rows, dim, io, res, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 7919 + rows * 31 + dim)
    x = (torch.randn(rows, dim + pad, generator=g) * 2).to(lc.IO[io])
    w = 1 + 0.3 * torch.randn(dim, generator=g)
    r = None if res is None else (3 * torch.randn(rows, dim, generator=g)).to(lc.IO[res])
    return x, w, r


def dev(t):
    return None if t is None else t.cuda()


def norm_slack(y, dim):
    # r: 1 rounding; the mean of squares dim + 4, halved by the root; rsqrt 4;
    # three products
    return (dim / 2 + 12) * lc.U32 * y.abs()


SHAPES = [(1, 1), (3, 7), (5, 64), (2, 127), (2, 128), (9, 129), (4, 512), (3, 513), (33, 1537),
          (2, 8192), (2, 8200), (1, 20000), (1, 32768)]


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("bf16", "bf16"), ("f32", None), ("f32", "f32"),
                                    ("f32", "bf16"), ("bf16", None)])
def test_forward(rows, dim, io, res):
    import selective_state_space_52_amd as m
    x, w, r = inputs(rows, dim, io, res)
    out, stream, rstd = m.rms_norm_fwd(x.cuda(), w.cuda(), residual=dev(r), eps=EPS, want_rstd=True)
    y, rr, rs = lc.rms_norm(x, w, r, EPS)
    lc.bound(out, y, norm_slack(y, dim), lc.IO[io])
    lc.bound(rstd, rs, (dim / 2 + 10) * lc.U32 * rs, torch.float32)
    if res is None:
        assert stream is None
    else:
        lc.bound(stream, rr, lc.U32 * rr.abs(), lc.IO[res])


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("f32", None)])
def test_forward_fp8(rows, dim, io, res):
    import selective_state_space_52_amd as m
    x, w, r = inputs(rows, dim, io, res, seed=1)
    q, scales, stream, rstd = m.rms_norm_fwd_fp8(x.cuda(), w.cuda(), residual=dev(r), eps=EPS)
    assert rstd is None and (stream is None) == (res is None)
    y, _, _ = lc.rms_norm(x, w, r, EPS)
    check_fp8(q, scales, y, norm_slack(y, dim))


def check_fp8(q, scales, y, slack):
    """q * scale is y to half a unit of e4m3, and the scale the smallest one."""
    codes = scales.view(torch.uint8).cpu()
    rows, dim = y.shape
    assert codes.shape == (rows, -(-dim // 128)) and q.shape == y.shape
    for j in range(codes.shape[1]):
        at = slice(128 * j, min(dim, 128 * j + 128))
        amax = y[:, at].abs().amax(1)
        off = slack[:, at].amax(1)
        s = lc.exp2i(codes[:, j])
        assert (amax <= 448 * s + off).all()
        assert ((amax >= 224 * s - off) | (codes[:, j] == 0)).all()
        got = q[:, at].cpu().double() * s[:, None]
        # 3 mantissa bits: half a unit is 2^-4 of the value, 2^-10 of the scale
        # below the normal range
        limit = y[:, at].abs() * 2.0 ** -4 + s[:, None] * 2.0 ** -10 + 1.07 * slack[:, at]
        assert ((got - y[:, at]).abs() <= limit).all()


def test_rows_of_zeros_and_extremes():
    import selective_state_space_52_amd as m
    x = torch.zeros(6, 300)
    x[1] = 1e-20
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 1e18
    x[5, 299] = -3.0
    w = torch.ones(300)
    out, _, _ = m.rms_norm_fwd(x.cuda(), w.cuda(), eps=EPS)
    y, _, _ = lc.rms_norm(x, w, None, EPS)
    assert (out[0] == 0).all()
    lc.bound(out[[0, 1, 4, 5]], y[[0, 1, 4, 5]], norm_slack(y[[0, 1, 4, 5]], 300), torch.float32)
    # an infinity gives 0 * inf at its place and zeros beside it; a NaN its whole row
    assert torch.isnan(out[2, 5]) and (out[2, :5] == 0).all()
    assert torch.isnan(out[3]).all()
    q, scales, _, _ = m.rms_norm_fwd_fp8(x.cuda(), w.cuda(), eps=EPS)
    assert (q[0].float() == 0).all() and (scales[0].view(torch.uint8) == 0).all()
    assert torch.isnan(q[2, 5].float()) and (q[2, :5].float() == 0).all()
    assert torch.isnan(q[3].float()).all()


def test_strided_rows_and_unaligned():
    import selective_state_space_52_amd as m
    x, w, r = inputs(17, 257, "bf16", "bf16", seed=3, pad=8)
    view = x.cuda()[:, 3:260]
    got, _, _ = m.rms_norm_fwd(view, w.cuda(), residual=r.cuda(), eps=EPS)
    same, _, _ = m.rms_norm_fwd(view.contiguous(), w.cuda(), residual=r.cuda(), eps=EPS)
    assert torch.equal(got, same)


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (700, 64), (9, 129), (1300, 513), (1500, 1537),
                                      (2, 8200), (1, 32768)])
@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("f32", None), ("bf16", "bf16"), ("f32", "f32")])
def test_backward(rows, dim, io, res):
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(rows + dim)
    r = (2 * torch.randn(rows, dim, generator=g)).to(lc.IO[res or io])
    dout = torch.randn(rows, dim, generator=g).to(lc.IO[io])
    w = 1 + 0.3 * torch.randn(dim, generator=g)
    rstd = (1 / torch.sqrt(r.double().square().mean(1) + EPS)).float()
    ds = None if res is None else torch.randn(rows, dim, generator=g).to(r.dtype)
    dx, dr, dw = m.rms_norm_bwd(dout.cuda(), r.cuda(), w.cuda(), rstd.cuda(), dresidual=dev(ds))
    again = m.rms_norm_bwd(dout.cuda(), r.cuda(), w.cuda(), rstd.cuda(), dresidual=dev(ds))
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[2])
    want, want_dw = lc.rms_norm_bwd(dout, r, w, rstd, ds)
    s, xhat = rstd.double()[:, None], r.double() * rstd.double()[:, None]
    wg = w.double() * dout.double()
    mean = (wg * xhat).abs().mean(1, keepdim=True)
    slack = lc.U32 * (s * (xhat.abs() * mean * (dim + 8) + 4 * wg.abs()) +
                      (0 if ds is None else 2 * ds.double().abs()))
    lc.bound(dx, want, slack, lc.IO[io])
    if res is None:
        assert dr is None
    else:
        lc.bound(dr, want, slack, lc.IO[res])
    lc.bound(dw, want_dw, (rows + 8) * lc.U32 * (dout.double() * xhat).abs().sum(0), torch.float32)


def test_backward_against_differences():
    """Central differences of the 64-bit forward along random directions."""
    import selective_state_space_52_amd as m
    rows, dim, h = 5, 200, 1e-5
    x, w, r = inputs(rows, dim, "f32", "f32", seed=5)
    g = torch.Generator().manual_seed(9)
    dout, ds = torch.randn(rows, dim, generator=g), torch.randn(rows, dim, generator=g)
    _, stream, rstd = m.rms_norm_fwd(x.cuda(), w.cuda(), residual=r.cuda(), eps=EPS, want_rstd=True)
    dx, dr, dw = m.rms_norm_bwd(dout.cuda(), stream, w.cuda(), rstd, dresidual=ds.cuda())
    assert torch.equal(dx, dr)

    def loss(xx, ww):
        y, rr, _ = lc.rms_norm(xx, ww, r, EPS)
        return float((y * dout.double()).sum() + (rr * ds.double()).sum())
    for k in range(4):
        vx = torch.randn(rows, dim, generator=g, dtype=torch.float64)
        vw = torch.randn(dim, generator=g, dtype=torch.float64)
        diff = (loss(x.double() + h * vx, w.double() + h * vw) -
                loss(x.double() - h * vx, w.double() - h * vw)) / (2 * h)
        grad = float((dx.cpu().double() * vx).sum() + (dw.cpu().double() * vw).sum())
        # terms of the two sums at fp32's rounding, and the differences' h^2
        size = float((dx.cpu().double() * vx).abs().sum() + (dw.cpu().double() * vw).abs().sum())
        assert abs(diff - grad) <= (dim * lc.U32 + 1e-6) * size


def test_other_stream_and_refusals():
    import selective_state_space_52_amd as m
    x, w, r = inputs(64, 640, "bf16", "f32", seed=2)
    base = m.rms_norm_fwd_fp8(x.cuda(), w.cuda(), residual=r.cuda())
    xs, ws, rs = x.cuda(), w.cuda(), r.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = m.rms_norm_fwd_fp8(xs, ws, residual=rs)
    side.synchronize()
    assert torch.equal(base[0].view(torch.uint8), other[0].view(torch.uint8))
    assert torch.equal(base[2], other[2])
    with pytest.raises(ValueError):
        m.rms_norm_fwd(x, w)                                   # CPU tensors
    with pytest.raises(ValueError):
        m.rms_norm_fwd(xs.half(), ws)
    with pytest.raises(ValueError):
        m.rms_norm_fwd(xs, ws[:-1].contiguous())
    with pytest.raises(ValueError):
        m.rms_norm_fwd(xs, ws, residual=rs[:32])
    with pytest.raises(ValueError):
        m.rms_norm_fwd(xs.t(), ws)
    with pytest.raises(m.MssmError):
        m.rms_norm_fwd(xs, ws, eps=-1.0)
    with pytest.raises(m.MssmError):
        m.rms_norm_fwd(torch.zeros(1, 40000, device="cuda"), torch.zeros(40000, device="cuda"))
    with pytest.raises(m.MssmError):
        m.rms_norm_fwd(torch.zeros(0, 64, device="cuda"), torch.zeros(64, device="cuda"))
