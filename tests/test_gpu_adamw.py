"""The AdamW step of many tensors against 64-bit references, states in fp32 and
in 8 bits."""
import math

import pytest
import torch

from tests import layer_common as lc
from tests import train_common as tc

pytestmark = pytest.mark.gpu
U32 = lc.U32
B1, B2, EPS, LR = 0.9, 0.97, 1e-8, 1e-2
SIZES = [1, 7, 127, 128, 129, 2048, 4095, 4096, 4097, 20000, 3]


def offsets(sizes):
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // 128) * 128)
    return at


def inputs(sizes, grad="mixed", seed=0, shift=0):
    """Tensors one after another in a flat buffer (so at any alignment), their
    gradients, and states as a run would have left them (in fp32)."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(sum(sizes) + shift, generator=g)
    params = list(flat[shift:].split(sizes))
    grads = []
    for i, n in enumerate(sizes):
        x = torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
        grads.append(x.bfloat16() if grad == "bf16" or (grad == "mixed" and i % 2) else x)
    at = offsets(sizes)
    m, v = torch.zeros(at[-1]), torch.zeros(at[-1])
    for n, a in zip(sizes, at):
        m[a:a + n] = 0.5 * torch.randn(n, generator=g)
        v[a:a + n] = torch.exp(2 * torch.randn(n, generator=g))
    return flat, params, grads, m, v


def on_gpu(flat, params, grads, shift=0):
    flat = flat.cuda()
    return flat, list(flat[shift:].split([len(p) for p in params])), [x.cuda() for x in grads]


def param_slack(want, old, m, v, step, lr, decay):
    """Roundings of the update: 2 of m, 3 of v (halved by its root), the root, the
    two corrections (and their own), eps, the reciprocal (4), the products: 16 of
    the update, and 3 of the parameter's own."""
    hat = (m / (1 - B1 ** step)).abs() / (torch.sqrt(v / (1 - B2 ** step)) + EPS)
    return U32 * (16 * lr * hat + 3 * old.double().abs())


@pytest.mark.parametrize("sizes", [[1], [300], SIZES, [5 + 37 * i for i in range(150)]])
@pytest.mark.parametrize("grad,copies", [("f32", "none"), ("bf16", "all"), ("mixed", "some")])
@pytest.mark.parametrize("step", [1, 1000])
def test_fp32_states(sizes, grad, copies, step):
    import selective_state_space_52_amd as mssm
    for shift in (0, 1):
        flat, params, grads, m, v = inputs(sizes, grad, shift=shift)
        fd, pd, gd = on_gpu(flat, params, grads, shift)
        md, vd = m.cuda(), v.cuda()
        cd = None
        if copies != "none":
            cd = [torch.zeros(n, dtype=torch.bfloat16, device="cuda")
                  if copies == "all" or i % 3 == 0 else None for i, n in enumerate(sizes)]
        decay = [0.1 * (i % 2) for i in range(len(sizes))]
        mssm.adamw_step(pd, gd, md, vd, step=step, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay,
                        copies=cd, grad_scale=0.3)
        at = offsets(sizes)
        if shift:
            assert float(fd[0]) == float(flat[0])
        for i, n in enumerate(sizes):
            s = slice(at[i], at[i] + n)
            # the scale 0.3 and the betas are fp32
            want, wm, wv = tc.adamw(params[i], grads[i], m[s], v[s], step, LR, B1, B2, EPS, decay[i], 0.3)
            g = grads[i].double() * 0.3
            lc.bound(md[s], wm, U32 * (3 * B1 * m[s].double().abs() + 5 * (1 - B1) * g.abs()), torch.float32)
            lc.bound(vd[s], wv, U32 * (3 * B2 * v[s].double() + 8 * (1 - B2) * g * g), torch.float32)
            cancel = U32 * (3 * B1 * m[s].double().abs() + 5 * (1 - B1) * g.abs()) / (1 - B1 ** step)
            slack = param_slack(want, params[i], wm, wv, step, LR, decay[i]) + \
                LR * cancel / (torch.sqrt(wv / (1 - B2 ** step)) + EPS)
            lc.bound(pd[i], want, slack, torch.float32)
            if cd is not None and cd[i] is not None:
                assert torch.equal(cd[i], pd[i].bfloat16())
            assert (md[at[i] + n:at[i + 1]] == 0).all() and (vd[at[i] + n:at[i + 1]] == 0).all()


@pytest.mark.parametrize("sizes", [[1], [300], SIZES, [5 + 37 * i for i in range(150)]])
@pytest.mark.parametrize("grad", ["f32", "mixed"])
@pytest.mark.parametrize("shift", [0, 1])
def test_8_bit_states(sizes, grad, shift):
    import selective_state_space_52_amd as mssm
    flat, params, grads, m, v = inputs(sizes, grad, seed=1, shift=shift)
    fd, pd, gd = on_gpu(flat, params, grads, shift)
    md, vd, ms, vs = mssm.adamw_state(pd, bits=8)
    at = offsets(sizes)
    seed = 12345678901234567890
    # two steps: from zero states, then from what the first has left
    for step in (1, 2):
        before = [t.cpu() for t in (md, vd, ms, vs)]
        old = [p.cpu().clone() for p in pd]
        mssm.adamw_step(pd, gd, md, vd, step=step, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.05,
                        m_scales=ms, v_scales=vs, grad_scale=0.3, seed=seed)
        pm, pr = tc.values8(before[0], before[2]), tc.values8(before[1], before[3])
        for i, n in enumerate(sizes):
            s = slice(at[i], at[i + 1])
            g = torch.zeros(at[i + 1] - at[i])
            g[:n] = grads[i].float()
            p = torch.zeros_like(g)
            p[:n] = old[i]
            want, wm, wv = tc.adamw(p, g, pm[s], pr[s] ** 2, step, LR, B1, B2, EPS, 0.05, 0.3)
            gg = g.double() * 0.3
            # m's two terms may cancel; the values and the scale are each rounded once
            m_off = U32 * (4 * B1 * pm[s].abs() + 5 * (1 - B1) * gg.abs())
            slack = param_slack(want, p, wm, wv, step, LR, 0.05) + \
                LR * m_off / (1 - B1 ** step) / (torch.sqrt(wv / (1 - B2 ** step)) + EPS)
            lc.bound(pd[i], want[:n], slack[:n] * 1.1, torch.float32)
            um, uv = tc.dither(len(g), seed, step)
            # a cancelled m is off by more of itself, but by no more of its block's
            # largest than of its terms; only v has a slack relative to each value
            tc.check_rounded(vd[s].cpu(), vs[at[i] // 128:at[i + 1] // 128].cpu(), wv.sqrt(), 8 * U32, uv, True)
            fine = (m_off <= 12 * U32 * wm.abs()).reshape(-1, 128).all(1)
            if fine.any():
                pick = lambda t: t.reshape(-1, 128)[fine].reshape(-1)  # noqa: E731
                tc.check_rounded(pick(md[s].cpu()), ms[at[i] // 128:at[i + 1] // 128].cpu()[fine], pick(wm),
                                 12 * U32, pick(um), False)
            assert (md[s][n:].float() == 0).all() and (vd[s][n:].float() == 0).all()
            # every m within a unit of its value
            got = tc.values8(md[s].cpu(), ms[at[i] // 128:at[i + 1] // 128].cpu())
            unit = ms[at[i] // 128:at[i + 1] // 128].cpu().double().repeat_interleave(128) * 2.0 ** -9
            assert ((got - wm).abs() <= torch.maximum(wm.abs() / 8, unit) * 1.001 + m_off * 2).all()


def test_8_bit_states_keep_their_means():
    """A moment that falls by a thousandth in a step does fall: rounding to nearest
    would hold every value but its block's largest.  One block of fixed gradients:
    after n steps the mean over the elements of value / exact is 1 within six
    standard deviations: a step moves a value v off its grid by (1 - b)(v - v'),
    and the rounding's variance is at most that times its unit (v / 8): in all at
    most n (1 - b) v^2 / 8."""
    import selective_state_space_52_amd as mssm
    n, steps, b1, b2 = 128 * 64, 400, 0.995, 0.999
    g = torch.Generator().manual_seed(3)
    start = torch.rand(n, generator=g) * 0.9 + 0.1
    start[::128] = 1.0
    p, zero = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    md, vd, ms, vs = mssm.adamw_state([p], bits=8)
    # betas of 0 make the first step take the gradient as the moments
    mssm.adamw_step([p], [start.cuda()], md, vd, step=1, lr=0.0, betas=(0.0, 0.0), m_scales=ms, v_scales=vs)
    m0, r0 = tc.values8(md.cpu(), ms.cpu()), tc.values8(vd.cpu(), vs.cpu())
    for i in range(steps):
        mssm.adamw_step([p], [zero], md, vd, step=i + 2, lr=0.0, betas=(b1, b2), m_scales=ms, v_scales=vs,
                        seed=77)
    rest = (torch.arange(n) % 128) != 0
    for got, was, keep in ((tc.values8(md.cpu(), ms.cpu()), m0, b1 ** steps),
                           (tc.values8(vd.cpu(), vs.cpu()), r0, b2 ** (steps / 2))):
        ratio = (got / (was * keep))[rest]
        spread = math.sqrt(-math.log(keep) / 8 / int(rest.sum()))
        # relative to what it has become: a value's own spread stays, its mean falls
        assert abs(float(ratio.mean()) - 1) <= 6 * spread / keep + 1e-3
        assert float((got != was)[rest].double().mean()) > 0.99


def test_non_finite_and_tiny_gradients():
    """NaN and infinities stay in their element; a block of tiny values counts as
    zero in 8 bits."""
    import selective_state_space_52_amd as mssm
    for bits in (32, 8):
        p = torch.ones(384, device="cuda")
        g = torch.full((384,), 0.5, device="cuda")
        g[3], g[7] = float("nan"), float("inf")
        g[128:256] = 1e-35
        g[256:] = 0.0
        m, v, ms, vs = mssm.adamw_state([p], bits)
        mssm.adamw_step([p], [g], m, v, step=1, lr=0.1, m_scales=ms, v_scales=vs, weight_decay=0.0)
        bad = torch.zeros(384, dtype=torch.bool, device="cuda")
        bad[3] = bad[7] = True
        assert torch.equal(torch.isnan(p), bad) or torch.equal(~torch.isfinite(p), bad)
        ok = ~bad
        assert float((p[:128][ok[:128]] - 0.9).abs().max()) < 1e-6
        assert (p[256:] == 1.0).all() and torch.isfinite(p[128:]).all()
        mf, vf = m.float(), v.float()
        assert torch.isfinite(mf[ok]).all() and torch.isfinite(vf[ok]).all()
        if bits == 8:
            # squares below the smallest normal number: their roots are not
            g = torch.full((128,), 1e-19, device="cuda")
            q, one = mssm.adamw_state([g], 8), torch.ones(128, device="cuda")
            mssm.adamw_step([one], [g], q[0], q[1], step=1, lr=0.1, m_scales=q[2], v_scales=q[3])
            root = q[1].double() * q[3].double()
            # v is 1e-41, 7000 of the smallest steps: 2^-13 of it, and all are the
            # block's largest
            assert float((root / (1e-19 * math.sqrt(1e-3)) - 1).abs().max()) < 2.0 ** -12
            assert torch.isnan(mf[bad]).all() and torch.isnan(vf[bad]).all()
            assert torch.isfinite(ms).all() and torch.isfinite(vs).all()
            assert float(ms[1]) == 0.0 and (mf[128:256] == 0).all() and float(ms[2]) == 0.0


@pytest.mark.parametrize("bits", [32, 8])
def test_device_values_in_a_graph(bits):
    """lr, step and grad_scale on the device: a captured step reads them in every
    replay and does what the eager one does with the same numbers; replays with
    other work in between.  1 - beta^step is fp32 there: 3 roundings."""
    import selective_state_space_52_amd as mssm
    sizes = [1000, 77, 4100]
    flat, params, grads, m, v = inputs(sizes, "mixed", seed=4)
    a, b = on_gpu(flat, params, grads), on_gpu(flat, params, grads)
    sa, sb = mssm.adamw_state(a[1], bits), mssm.adamw_state(b[1], bits)
    lr, scale = torch.tensor([LR], device="cuda"), torch.tensor([0.5], device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def call(x, s, **o):
        mssm.adamw_step(x[1], x[2], s[0], s[1], betas=(B1, B2), m_scales=s[2], v_scales=s[3], seed=9, **o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, sa, step=step, lr=lr, grad_scale=scale)
    for k in range(1, 5):
        step.fill_(k)
        lr.fill_(LR / k)
        scale.fill_(0.5 + k)
        graph.replay()
        torch.cuda.synchronize()
        call(b, sb, step=k, lr=float(lr), grad_scale=float(scale))
        for x, y in zip(sa, sb):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        off = (a[0] - b[0]).abs().cpu().double()
        # each of k steps moves a parameter by lr / k or so times 10 at most
        assert (off <= U32 * (a[0].cpu().double().abs() * 2 * k + 8 * 10 * LR * k)).all()


def test_a_tensor_past_32_bits():
    """More than 2^31 elements behind a small tensor: the last ones are stepped, and
    by fractions of their own."""
    import selective_state_space_52_amd as mssm
    n = (1 << 31) + 4000
    small = torch.ones(5, device="cuda")
    p = torch.ones(n, device="cuda")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-1], g[-200] = -0.25, 0.125
    m, v, ms, vs = mssm.adamw_state([small, p], 8)
    mssm.adamw_step([small, p], [torch.ones(5, device="cuda"), g], m, v, step=1, lr=0.1, m_scales=ms,
                    v_scales=vs, weight_decay=0.0, seed=5)
    # the first step moves by lr against the gradient's sign, whatever its size
    for at, sign in ((0, 1), (1 << 31, 1), (n - 1, -1), (n - 200, 1), (n - 2, 1)):
        assert abs(float(p[at]) - (1 - 0.1 * sign)) < 1e-6
    assert abs(float(p[::1 << 20].double().mean()) - 0.9) < 1e-6
    end = 128 + n
    got = m[128:][n - 200].double() * ms[(end - 200) // 128].double()
    assert abs(float(got) / 0.0125 - 1) <= 0.125 and float(ms[-1]) > 0
    assert (m[end:].float() == 0).all()


def test_other_stream_and_repeat():
    import selective_state_space_52_amd as mssm
    flat, params, grads, m, v = inputs(SIZES, seed=6)
    got = []
    for k in range(3):
        x = on_gpu(flat, params, grads)
        s = mssm.adamw_state(x[1], 8)
        side = torch.cuda.Stream() if k == 1 else torch.cuda.current_stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for step in (1, 2, 3):
                mssm.adamw_step(x[1], x[2], s[0], s[1], step=step, lr=LR, m_scales=s[2], v_scales=s[3])
        side.synchronize()
        got.append((x[0], *(t.view(torch.uint8) for t in s)))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_refusals():
    import selective_state_space_52_amd as mssm
    p, g = torch.zeros(4, 100, device="cuda"), torch.zeros(4, 100, device="cuda")
    m, v, _, _ = mssm.adamw_state([p])
    m8, v8, ms, vs = mssm.adamw_state([p], 8)

    def call(params=None, grads=None, mm=m, vv=v, **o):
        mssm.adamw_step([p] if params is None else params, [g] if grads is None else grads, mm, vv,
                        **{**dict(step=1, lr=0.1), **o})
    for bad in (dict(params=[]), dict(grads=[]), dict(params=[p.bfloat16()]), dict(params=[p.t()]),
                dict(grads=[g.half()]), dict(grads=[g[:3]]), dict(grads=[g.t().contiguous().t()]),
                dict(grads=[g.cpu()]), dict(mm=m[:-128]), dict(vv=v8), dict(m_scales=ms),
                dict(mm=m8, vv=v8), dict(mm=m8, vv=v8, m_scales=ms, v_scales=vs[:-1]),
                dict(copies=[]), dict(copies=[p]), dict(weight_decay=[0.1, 0.2]),
                dict(lr=torch.zeros(2, device="cuda")), dict(step=torch.zeros(1, device="cuda")),
                dict(grad_scale=torch.zeros(1, dtype=torch.float64, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    two = mssm.adamw_state([p, p])
    for bad in (dict(step=0), dict(betas=(1.0, 0.9)), dict(eps=-1.0),
                dict(params=[p, p], grads=[g, g], mm=two[0], vv=two[1]),      # the same tensor twice
                dict(grads=[p])):
        with pytest.raises(mssm.MssmError):
            call(**bad)
    empty = torch.zeros(0, device="cuda")
    with pytest.raises(mssm.MssmError):
        call(params=[p, empty], grads=[g, empty])
