"""The Mamba-2 single-token step with its convolution, against the 64-bit
recurrence and against the prompt's scan."""
import pytest
import torch

from tests import layer_common as lc

pytestmark = pytest.mark.gpu


def inputs(batch, heads, groups, N, io, width=4, cache=None, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 101 + batch * 7 + heads)
    cache = cache or batch
    dim, dt = heads * 64, lc.IO[io]
    ch = dim + 2 * groups * N
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(state=0.2 * r(cache, dim, N), conv_state=r(cache, ch, width - 1).to(dt),
                xbc=r(batch, ch + pad).to(dt)[:, :ch], dt=r(batch, heads + pad).to(dt)[:, :heads],
                conv_weight=0.5 * r(ch, width), A=-1 - 15 * torch.rand(heads, generator=g),
                conv_bias=0.1 * r(ch), D=r(heads), z=r(batch, dim + pad).to(dt)[:, :dim],
                dt_bias=r(heads) - 3, softplus=True, ngroups=groups, slots=None)


def on_gpu(a):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}


def check(a, io):
    import selective_state_space_52_amd as m
    want = lc.mamba2_step(**a)
    size = lc.mamba2_step(**a, sizes=True)
    d = on_gpu(a)
    for k in ("xbc", "dt", "z"):   # keep the rows' strides
        if a[k] is not None:
            d[k] = torch.empty_strided(a[k].shape, a[k].stride(), dtype=a[k].dtype, device="cuda")
            d[k].copy_(a[k])
    got = m.mamba2_state_update(**d)
    N = a["state"].shape[2]
    # the exponent dt A is at most about 16 * 8 with 3 roundings of its own
    slack = 512 * lc.U32
    lc.bound(d["state"], want[1], slack * size[1], torch.float32)
    lc.bound(got, want[0], (slack + N * lc.U32) * size[0], lc.IO[io])
    assert torch.equal(d["conv_state"].cpu().double(), want[2])


@pytest.mark.parametrize("batch,heads,groups,N", [(1, 1, 1, 64), (1, 24, 1, 128), (3, 4, 2, 64),
                                                  (5, 6, 3, 128), (64, 24, 1, 64)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_step(batch, heads, groups, N, io, width):
    check(inputs(batch, heads, groups, N, io, width), io)


@pytest.mark.parametrize("drop", ["conv_bias", "D", "z", "dt_bias", "softplus"])
def test_without(drop):
    a = inputs(4, 3, 1, 128, "bf16")
    a[drop] = False if drop == "softplus" else None
    check(a, "bf16")


def test_strided_rows():
    check(inputs(5, 4, 2, 128, "bf16", pad=3), "bf16")
    check(inputs(2, 3, 1, 64, "f32", pad=1), "f32")


def test_slots():
    a = inputs(6, 4, 1, 128, "bf16", cache=9)
    a["slots"] = torch.tensor([8, 0, -1, 3, 9, 2], dtype=torch.int32)   # -1, 9: padding
    check(a, "bf16")
    a = inputs(2, 4, 1, 128, "f32", cache=70)
    a["slots"] = torch.tensor([69, 0], dtype=torch.int32)
    check(a, "f32")


def test_extreme_steps():
    """Steps of zero (the state stays), huge ones (it is replaced) and a
    non-finite state in another sequence's row."""
    a = inputs(3, 2, 1, 64, "f32")
    a["softplus"], a["dt_bias"] = False, None
    a["dt"] = torch.tensor([[0.0, 0.0], [100.0, 100.0], [1.0, 1.0]])
    check(a, "f32")
    a["state"][2, 0, 0] = float("nan")
    import selective_state_space_52_amd as m
    d = on_gpu(a)
    out = m.mamba2_state_update(**d)
    bad = torch.isnan(out.cpu())
    assert bad[2, 0] and bad.sum() == 1


def test_continues_a_prompt():
    """Prompt through the convolution and the scan, then the step: the same as
    the prompt one token longer."""
    import selective_state_space_52_amd as m
    batch, L, heads, groups, N = 2, 70, 3, 1, 128
    dim, ch = heads * 64, heads * 64 + 2 * groups * N
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    xbc, dt, z = (r(batch, L + 1, n).bfloat16() for n in (ch, heads, dim))
    w, b, A, D = 0.4 * r(ch, 4), 0.1 * r(ch), -1 - r(heads).abs(), r(heads)
    bias = r(heads) - 3

    def prompt(n):
        u = m.causal_conv1d_fwd(xbc[:, :n].contiguous(), w, b, layout="bld")
        x, B, C = (t.contiguous() for t in u.split([dim, groups * N, groups * N], dim=2))
        last = torch.zeros(batch, dim, N, device="cuda")
        out = m.mamba2_scan_fwd(x.view(batch, n, heads, 64), dt[:, :n].contiguous(), A,
                                B.view(batch, n, groups, N), C.view(batch, n, groups, N), D=D,
                                z=z[:, :n].contiguous().view(batch, n, heads, 64), dt_bias=bias,
                                last_state=last)
        return out.reshape(batch, n, dim), last
    _, state = prompt(L)
    conv_state = xbc[:, L - 3:L].transpose(1, 2).contiguous()
    out = m.mamba2_state_update(state, conv_state, xbc[:, L], dt[:, L], w, A, conv_bias=b, D=D,
                                z=z[:, L], dt_bias=bias)
    want, want_state = prompt(L + 1)
    # the prompt rounds the convolution's output, and its scan's operands, to bf16
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    assert rel(out, want[:, L]) < 0.02 and rel(state, want_state) < 0.01
    assert torch.equal(conv_state, xbc[:, L - 2:L + 1].transpose(1, 2))


def test_refusals():
    import selective_state_space_52_amd as m
    good = on_gpu(inputs(2, 2, 1, 64, "bf16"))

    def bad(**o):
        with pytest.raises(ValueError):
            m.mamba2_state_update(**{**good, **o})
    bad(state=good["state"].cpu())
    bad(state=good["state"][:1].contiguous())
    bad(conv_state=good["conv_state"].float())
    bad(xbc=good["xbc"][:, :-1].contiguous())
    bad(A=good["A"][:1].contiguous())
    bad(ngroups=2)
    bad(slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    bad(out=torch.empty(2, 2, device="cuda"))
    bad(dt=good["dt"].t().contiguous().t()[:1].expand(2, 2))
    a = on_gpu(inputs(2, 2, 1, 64, "bf16"))
    with pytest.raises(m.MssmError):     # N = 32
        m.mamba2_state_update(**{**a, "state": a["state"][..., :32].contiguous(),
                                 "xbc": a["xbc"][:, :192].contiguous(),
                                 "conv_state": a["conv_state"][:, :192].contiguous(),
                                 "conv_weight": a["conv_weight"][:192].contiguous(),
                                 "conv_bias": a["conv_bias"][:192].contiguous()})
