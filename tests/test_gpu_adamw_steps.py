"""The AdamW step where it repeats itself or its numbers are at their type's ends."""
import pytest
import torch

from tests import layer_common as lc
from tests import train_common as tc
from tests.test_gpu_adamw import offsets

pytestmark = pytest.mark.gpu
U32 = lc.U32


def states(mssm, params, bits):
    m, v, ms, vs = mssm.adamw_state(params, bits)
    return (m, v), dict(m_scales=ms, v_scales=vs)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-8])
def test_squares_below_the_normal_numbers(bits, eps):
    """Gradients of 1e-19: v is 1e-41, whose root is 3e-21.  The step is lr g / (|g| +
    eps) with it, and neither lr g / eps nor an infinity.

    The square, 1e-38, and v are each rounded to a multiple of 2^-149, so v is off by
    2^-150 (1 + 1e-3), the step by half of that relative to v, and 8 roundings."""
    import selective_state_space_52_amd as mssm
    g = torch.full((300,), 1e-19, device="cuda")
    g[1::2] *= -1
    g[5], g[200] = 0.5, -2.0                    # beside ordinary ones
    p = torch.ones(300, device="cuda")
    mv, scales = states(mssm, [p], bits)
    mssm.adamw_step([p], [g], *mv, step=1, lr=0.1, eps=eps, weight_decay=0.0, **scales)
    gd = g.double().cpu()
    want = 1.0 - 0.1 * gd / (gd.abs() + eps)
    off = 0.1 * (2.0 ** -150 * 1.001 / 1e-41 / 2 + 8 * U32)
    assert float((p.double().cpu() - want).abs().max()) <= off + U32


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-30, 1e-40, 1e-300])
def test_an_eps_below_the_normal_numbers(bits, eps):
    """A gradient of 0 moves nothing, however small eps is: 0 / eps is 0."""
    import selective_state_space_52_amd as mssm
    p, g = torch.ones(300, device="cuda"), torch.zeros(300, device="cuda")
    g[7] = 3.0
    mv, scales = states(mssm, [p], bits)
    for step in (1, 2):
        mssm.adamw_step([p], [g], *mv, step=step, lr=0.25, eps=eps, weight_decay=0.0, **scales)
    assert abs(float(p[7]) - 0.5) <= 0.25 * 2.0 ** -3        # 8 bits round its moments
    p[7] = 1.0
    assert (p == 1.0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [float("inf"), float("nan")])
@pytest.mark.parametrize("on_device", [False, True])
def test_what_lies_between_tensors_stays_zero(bits, scale, on_device):
    """Also where the gradients' scale is not finite (a loss scale that overflowed):
    0 * infinity is no element's."""
    import selective_state_space_52_amd as mssm
    sizes = [1, 126, 127, 128, 130, 1023, 4097]
    p = [torch.ones(n, device="cuda") for n in sizes]
    mv, scales = states(mssm, p, bits)
    value = torch.tensor([scale], device="cuda") if on_device else scale
    mssm.adamw_step(p, [torch.ones_like(x) for x in p], *mv, step=1, lr=0.1, grad_scale=value, **scales)
    at = offsets(sizes)
    for t in mv:
        t = t.float()
        for n, a, b in zip(sizes, at, at[1:]):
            assert (t[a + n:b] == 0).all() and not torch.isfinite(t[a:a + n]).any()
    assert not any(torch.isfinite(x).any() for x in p)
    assert all(s is None or (s == 0).all() for s in scales.values())


def near_root(x):
    """The nearest fp32 root (torch's own on the CPU is a unit off at places).  One
    rounded to 53 bits first is at least 2 * 24 + 2 bits wide: the second rounding
    changes nothing."""
    return x.double().sqrt().float()


def to_8_bits(x, u, positive):
    """The definition in fp32, each operation of these tensors rounded once."""
    x, u = x.view(-1, 128), u.view(-1, 128)
    one, limit = torch.ones(1), torch.full((1,), 448.0)
    most = x.abs().amax(1, keepdim=True)
    most = torch.where(most < 2.0 ** -100, 0.0, most)
    y = x * torch.where(most > 0, limit * (one / most), 0.0)
    unit = torch.exp2(torch.frexp(y)[1].sub(1).clamp(min=-6).double() - 3).float()
    value = torch.minimum(torch.floor(y.abs() / unit + u) * unit, limit)
    if positive:
        value = torch.where((value == 0) & (y > 0), 2.0 ** -9, value)
    return torch.copysign(value, y).to(lc.F8).flatten(), (most * (one / limit)).flatten()


class Definition:
    """The states' definition, one tensor after another."""

    def __init__(self, sizes, bits, b1, b2):
        self.sizes, self.at, self.bits = sizes, offsets(sizes), bits
        n = self.at[-1]
        self.m, self.v = torch.zeros(n), torch.zeros(n)           # v: its root in 8 bits
        if bits == 8:
            self.m, self.v = self.m.to(lc.F8), self.v.to(lc.F8)
            self.m_scales, self.v_scales = torch.zeros(n // 128), torch.zeros(n // 128)
        self.betas = torch.tensor([b1, b2], dtype=torch.float64)

    def step(self, grads, scale, seed, step):
        """Returns the moments before they go to 8 bits."""
        b1, b2 = self.betas.float()
        r1, r2 = (1.0 - self.betas).float()
        g = torch.zeros(self.at[-1])
        um, uv = torch.zeros(self.at[-1]), torch.zeros(self.at[-1])
        for n, a, b, grad in zip(self.sizes, self.at, self.at[1:], grads):
            g[a:a + n] = grad.float() * torch.tensor(scale)
            low, high = tc.dither(b - a, seed, step)
            um[a:b], uv[a:b] = low.float() * 2.0 ** -24, high.float() * 2.0 ** -24
        m, v = self.m, self.v
        if self.bits == 8:
            m = m.float() * self.m_scales.repeat_interleave(128)
            v = v.float() * self.v_scales.repeat_interleave(128)
            v = v * v
        m = m * b1 + g * r1
        v = v * b2 + (g * g) * r2
        if self.bits == 8:
            self.m, self.m_scales = to_8_bits(m, um, False)
            self.v, self.v_scales = to_8_bits(near_root(v), uv, True)
        else:
            self.m, self.v = m, v
        return m, v

    def same(self, mv, scales):
        got = list(mv) + [s for s in scales.values() if s is not None]
        want = [self.m, self.v] + ([self.m_scales, self.v_scales] if self.bits == 8 else [])
        return all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def gradients(kind, sizes, g):
    out = []
    for i, n in enumerate(sizes):
        x = torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
        if kind == "rare":            # most elements' moments only fall
            x *= torch.rand(n, generator=g) < 0.05
        elif kind == "wide":          # from 2^-100 up, blocks of tiny values among them
            x *= torch.exp2(-100 * torch.rand(n // 64 + 1, generator=g)).repeat_interleave(64)[:n]
        out.append(x.bfloat16() if i % 2 else x)
    return out


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kind", ["plain", "rare", "wide"])
@pytest.mark.parametrize("betas", [(0.9, 0.95), (0.9, 0.999)])
def test_states_over_many_steps(bits, kind, betas):
    """30 steps in a row leave the states that the definition gives, to the last bit:
    what differs once would move values by whole units later.  Parameters: each step
    from the step's own start, 16 roundings of the update (of moments whose terms
    cancel, of those terms), 3 of the parameter."""
    import selective_state_space_52_amd as mssm
    sizes = [1, 127, 129, 4097, 60000, 3]
    seed, scale, lr, eps = 0xFEDCBA9876543210, 0.7, 1e-2, 1e-8
    g = torch.Generator().manual_seed(17)
    p = [torch.randn(n, generator=g).cuda() for n in sizes]
    mv, scales = states(mssm, p, bits)
    want = Definition(sizes, bits, *betas)
    for step in range(1, 31):
        grads = gradients(kind, sizes, g)
        old = torch.cat(p).double().cpu()
        before = want.m.double() * want.m_scales.double().repeat_interleave(128) if bits == 8 else want.m.double()
        mssm.adamw_step(p, [x.cuda() for x in grads], *mv, step=step, lr=lr, betas=betas, eps=eps,
                        weight_decay=0.1, grad_scale=scale, seed=seed, **scales)
        m, v = want.step(grads, scale, seed, step)
        assert want.same(mv, scales), step
        here = torch.cat([torch.arange(a, a + n) for n, a in zip(sizes, want.at)])
        by = torch.sqrt(v.double()[here] / (1 - betas[1] ** step)) + eps
        terms = before[here].abs() * betas[0] + (1 - betas[0]) * scale * torch.cat(
            [x.double() for x in grads]).abs()
        update = m.double()[here] / (1 - betas[0] ** step) / by
        slack = U32 * (16 * lr * terms / (1 - betas[0] ** step) / by + 3 * old.abs())
        lc.bound(torch.cat(p), old * (1 - lr * 0.1) - lr * update, slack, torch.float32)
