"""Log-probabilities of tokens, the policy and the preference loss, and their
gradients, against 64-bit references."""
import pytest
import torch

from tests import layer_common as lc
from tests import train_common as tc

pytestmark = pytest.mark.gpu
U32 = lc.U32
SHAPES = [(1, 1), (3, 2), (3, 7), (2, 8), (5, 9), (4, 511), (3, 8192), (2, 8193), (2, 16385), (3, 50257),
          (2, 65536), (1, 65537), (1, 70001), (2, 131073),
          (1, 300007), (5, 65535), (3, 73727)]


def inputs(rows, vocab, io, seed=0, pad=0, skip=True):
    g = torch.Generator().manual_seed(seed * 101 + rows * 31 + vocab)
    wide = torch.randn(rows, vocab + pad, generator=g) * 3
    wide[:, ::97] += 6
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    if skip and rows > 1:
        tokens[rows // 2] = -1
    if skip and rows > 3:
        tokens[0] = vocab
    return wide.to(lc.IO[io]), tokens, g


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("io,t", [("bf16", 1.0), ("f32", 1.0), ("f32", 0.3)])
def test_logprobs(rows, vocab, io, t):
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(rows, vocab, io)
    logp, stats = m.token_logprobs_fwd(logits.cuda(), tokens.cuda(), temperature=t)
    want, top, log_sum, p = tc.logprobs(logits, tokens, t)
    slack, of_sum, of_p = tc.logprob_slack(logits, tokens, t)
    live = (tokens >= 0) & (tokens < vocab)
    lc.bound(logp[live], want[live], slack[live], torch.float32)
    assert (logp.cpu()[~live] == 0).all()
    assert torch.equal(stats[:, 0].cpu()[live], top[live].float())
    lc.bound(stats[:, 1][live], log_sum[live], of_sum[live], torch.float32)
    # back, with a row of slope zero
    d = torch.randn(rows, generator=g)
    if rows > 2:
        d[-1] = 0.0
    got = m.token_logprobs_bwd(logits.cuda(), tokens.cuda(), stats, d.cuda(), temperature=t)
    factor = torch.where(live, d.double() / t, 0.0)
    check_slope(got, p, tokens, factor, of_p, lc.IO[io])


def check_slope(got, p, tokens, factor, of_p, dtype, of_factor=0.0):
    """factor ([j = token] - p): p is off by of_p of itself, factor by 4 U32 (and
    of_factor) of it."""
    want = tc.softmax_slope(p, tokens, factor)
    f = factor.abs()[:, None]
    own = torch.zeros_like(p)
    for i, t in enumerate(tokens.tolist()):
        if 0 <= t < p.shape[1]:
            own[i, t] = 1.0
    # the hardware exp2 gives 0 for what lies below the smallest normal number
    slack = f * p * of_p + (4 * U32 + of_factor) * f * (p + own) + f * 2.0 ** -126
    lc.bound(got, want, slack, dtype)
    assert (got.cpu()[factor == 0] == 0).all()


POLICY = [(1, 1), (6, 9), (7, 511), (5, 8193), (4, 50257), (2, 70001), (3, 131073)]


@pytest.mark.parametrize("rows,vocab", POLICY)
@pytest.mark.parametrize("io,t,kl,low,high", [("bf16", 1.0, 0.05, 0.2, 0.2), ("f32", 0.7, 0.0, 0.1, 0.3),
                                              ("f32", 1.0, 0.3, 0.2, 0.28)])
@pytest.mark.parametrize("where", ["inside", "above", "below", "mixed"])
def test_policy(rows, vocab, io, t, kl, low, high, where):
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(rows, vocab, io, seed=1)
    logp, _, _, p = tc.logprobs(logits, tokens, t)
    moved = {"inside": torch.full((rows,), 0.03), "above": torch.full((rows,), 0.5),
             "below": torch.full((rows,), -0.6), "mixed": 0.9 * (torch.arange(rows) % 3 - 1)}[where]
    old = (logp - moved).float()
    adv, w = torch.randn(rows, generator=g), torch.rand(rows, generator=g)
    ref = (logp + 0.4 * torch.randn(rows, generator=g)).float() if kl else None
    if rows > 2:
        w[-1] = 0.0
    slack, _, of_p = tc.logprob_slack(logits, tokens, t)
    args = [logits.cuda(), tokens.cuda(), old.cuda(), adv.cuda()]
    more = dict(ref_logprobs=None if ref is None else ref.cuda(), weights=w.cuda(), temperature=t,
                clip_low=low, clip_high=high, kl_coef=kl)
    loss, got_logp, grad = m.policy_loss(*args, **more)
    want, slope = tc.policy(logp, tokens, vocab, old, adv, ref, low, high, kl)
    lc.bound(got_logp, logp, slack, torch.float32)
    # an exponential of something off by e is off by e of itself, and 4 U32; the
    # clip's edges are fp32
    off = slack + 2 * U32 * logp.abs() + 8 * U32
    ratio = torch.exp(logp - old.double())
    size = ratio * adv.double().abs()
    kl_size = 0.0 if ref is None else kl * (torch.exp(ref.double() - logp) + 1)
    lc.bound(loss, want, off * (size + kl_size) + 4 * U32 * (adv.double().abs() * 1.4 + kl_size),
             torch.float32)
    factor = slope * w.double() / t
    of_factor = (off * (size + kl_size) * w.double() / t / factor.abs().clamp(min=1e-300))[:, None]
    check_slope(grad, p, tokens, factor, of_p, lc.IO[io], of_factor)
    # without the gradient, without weights, and in place: the same bits
    only, lp, none = m.policy_loss(*args, **more, want_grad=False)
    assert none is None and torch.equal(only, loss) and torch.equal(lp, got_logp)
    place = logits.cuda()
    l2, _, g2 = m.policy_loss(place, *args[1:], **more, out=place)
    assert g2 is place and torch.equal(l2, loss) and torch.equal(place, grad)
    ones = m.policy_loss(*args, **{**more, "weights": torch.ones(rows, device="cuda")})
    free = m.policy_loss(*args, **{**more, "weights": None})
    assert all(torch.equal(a, b) for a, b in zip(ones, free))


def test_policy_on_the_clip():
    """Ratios of exactly 1 with no room to move: both sides of the min are equal,
    and the slope is the unclipped one's."""
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(6, 300, "f32", skip=False)
    ld, td = logits.cuda(), tokens.cuda()
    logp, stats = m.token_logprobs_fwd(ld, td)
    adv = torch.tensor([1.0, -2.0, 0.0, 0.5, 3.0, -1.0], device="cuda")
    loss, _, grad = m.policy_loss(ld, td, logp, adv, clip_low=0.0, clip_high=0.0)
    assert torch.equal(loss, -adv)
    assert torch.equal(grad, m.token_logprobs_bwd(ld, td, stats, -adv))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 9000, 70003])
def test_masked_logits(io, vocab):
    """-infinity and the type's lowest value among the logits, rows of nothing
    else, NaN and +infinity."""
    import selective_state_space_52_amd as m
    dtype = lc.IO[io]
    low = torch.finfo(dtype).min
    logits, tokens, g = inputs(9, vocab, io, seed=3, skip=False)
    tokens[:] = 5
    logits[0, 6:] = float("-inf")
    logits[1, :] = float("-inf")
    logits[1, 5] = 2.0                       # the only one left
    logits[2, 6:] = low
    logits[3, :] = low                       # an even distribution
    logits[4, 5] = float("-inf")             # the token itself
    logits[5, :] = float("-inf")             # nothing left
    logits[6, 7] = float("nan")
    logits[7, 7] = float("inf")
    tokens[8] = -1
    logits[8] = float("nan")                 # not read
    for t in (1.0, 0.5):
        logp, stats = m.token_logprobs_fwd(logits.cuda(), tokens.cuda(), temperature=t)
        want, _, _, p = tc.logprobs(logits, tokens, t)
        want[8] = 0.0
        fine = [0, 1, 2, 3]
        slack, _, of_p = tc.logprob_slack(logits[fine], tokens[fine], t)
        lc.bound(logp[fine], want[fine], slack, torch.float32)
        assert float(logp[1]) == 0.0 and float(logp[4]) == -torch.inf and float(logp[8]) == 0.0
        assert torch.isnan(logp[5:8]).all()
        d = torch.full((9,), 0.5)
        got = m.token_logprobs_bwd(logits.cuda(), tokens.cuda(), stats, d.cuda(), temperature=t).cpu()
        check_slope(got[fine], p[fine], tokens[fine], d.double()[fine] / t, of_p, dtype)
        assert (got[0, 6:] == 0).all() and (got[1] == 0).all() and (got[8] == 0).all()
        assert torch.isnan(got[5:8]).all() and torch.isfinite(got[4]).all() and float(got[4, 5]) == 0.5 / t
        # the loss in one read agrees, and its padding row's own entries are not read
        adv = -d                                    # slope 0.5 where the ratio is 1
        old = torch.where(torch.isfinite(logp.cpu()), logp.cpu(), 0.0)
        old[8] = adv[8] = float("nan")
        loss, lp, grad = m.policy_loss(logits.cuda(), tokens.cuda(), old.cuda(), adv.cuda(),
                                       temperature=t, clip_low=9.0, clip_high=9.0)
        assert torch.equal(lp[:5], logp[:5]) and float(loss[8]) == 0.0 and (grad[8] == 0).all()
        for i in fine:
            assert torch.equal(grad[i].cpu(), got[i])


@pytest.mark.parametrize("vocab,pad,first", [(1003, 5, 3), (8197, 11, 4), (40, 24, 1), (65535, 9, 1),
                                             (65536, 9, 1), (65536, 8, 3), (70001, 7, 2), (81919, 2, 1),
                                             (81920, 1, 1)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strided_rows(vocab, pad, first, io):
    """Views at any column of wider rows, gradients into such views and in place:
    the values of whole tensors (sums may be taken in another order where rows
    begin at an odd address), and nothing written beside them."""
    import selective_state_space_52_amd as m
    first = min(first, pad)
    wide, tokens, g = inputs(6, vocab, io, seed=4, pad=pad)
    wd, td = wide.cuda(), tokens.cuda()
    view = wd[:, first:first + vocab]
    plain = view.cpu().contiguous()
    logp, stats = m.token_logprobs_fwd(view, td)
    want, top, log_sum, p = tc.logprobs(plain, tokens, 1.0)
    slack, of_sum, of_p = tc.logprob_slack(plain, tokens, 1.0)
    live = (tokens >= 0) & (tokens < vocab)
    lc.bound(logp[live], want[live], slack[live], torch.float32)
    assert torch.equal(stats[:, 0].cpu()[live], top[live].float())
    d = torch.randn(6, generator=g)
    factor = torch.where(live, d.double(), 0.0)
    out = torch.full((6, vocab + 9), 7.0, dtype=lc.IO[io], device="cuda")
    got = m.token_logprobs_bwd(view, td, stats, d.cuda(), out=out[:, 2:2 + vocab])
    check_slope(got, p, tokens, factor, of_p, lc.IO[io])
    assert (out[:, :2] == 7).all() and (out[:, 2 + vocab:] == 7).all()     # nothing beside it
    out.fill_(7.0)
    # slope -adv = d where the ratio is 1
    again = m.policy_loss(view, td, logp, -d.cuda(), out=out[:, 2:2 + vocab])
    assert torch.equal(again[1], logp) and torch.equal(again[2], got)
    assert (out[:, :2] == 7).all() and (out[:, 2 + vocab:] == 7).all()
    keep = wd.clone()
    place = m.policy_loss(view, td, logp, -d.cuda(), out=view)
    assert torch.equal(place[2], got)
    keep[:, first:first + vocab] = got
    assert torch.equal(wd, keep)


def test_rows_taken_out():
    """A weight of 0 leaves nothing of a row or pair in the gradient, whatever its
    loss is; a KL term of weight 0 is none."""
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(6, 300, "f32", seed=7, skip=False)
    ld, td = logits.cuda(), tokens.cuda()
    logp, _ = m.token_logprobs_fwd(ld, td)
    adv = torch.randn(6, generator=g).cuda()
    old, w = logp.clone(), torch.ones(6, device="cuda")
    base = m.policy_loss(ld, td, old, adv, weights=w)[2]
    old[1], old[2], w[1], w[2] = float("nan"), float("-inf"), 0.0, -0.0
    ref = torch.full_like(old, float("-inf"))
    loss, _, grad = m.policy_loss(ld, td, old, adv, ref_logprobs=ref, weights=w, kl_coef=0.0)
    assert (grad[1:3] == 0).all() and torch.isnan(loss[1])
    keep = [0, 3, 4, 5]
    assert torch.equal(grad[keep], base[keep]) and torch.isfinite(loss[keep]).all()
    at = torch.tensor([0, 1, 3, 4, 6], dtype=torch.int32, device="cuda")
    _, d = m.preference_loss(old, logp, at, weights=torch.tensor([0.0, 1.0], device="cuda"))
    assert (d[:3] == 0).all() and (d[3:] != 0).all() and torch.isfinite(d).all()


def test_logits_past_32_bits():
    """Rows whose elements lie beyond 2^31."""
    import selective_state_space_52_amd as m
    rows, vocab = 43000, 50304
    logits = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    logits[-3:] = torch.randn(3, vocab, device="cuda").bfloat16() * 3
    tokens = torch.full((rows,), -1, device="cuda")
    tokens[-3:] = torch.tensor([5, 50303, 0], device="cuda")
    d = torch.ones(rows, device="cuda")
    few, t3 = logits[-3:].clone(), tokens[-3:].clone()
    logp, stats = m.token_logprobs_fwd(logits, tokens)
    want, want_stats = m.token_logprobs_fwd(few, t3)
    assert torch.equal(logp[-3:], want) and (logp[:-3] == 0).all()
    grad = m.token_logprobs_bwd(logits, tokens, stats, d)
    assert torch.equal(grad[-3:], m.token_logprobs_bwd(few, t3, want_stats, d[:3]))
    assert not grad[:-3].any()
    _, _, grad = m.policy_loss(logits, tokens, logp, -d, out=grad)
    assert torch.equal(grad[-3:], m.policy_loss(few, t3, want, -d[:3])[2]) and not grad[:-3].any()


def test_policy_gradient_against_differences():
    """Central differences of the 64-bit loss, away from the clip's corners."""
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(8, 60, "f32", seed=6)
    logp, _, _, _ = tc.logprobs(logits, tokens, 0.8)
    moved = torch.tensor([0.05, 0.6, -0.7, 0.02, -0.05, 0.5, -0.6, 0.01])
    old, adv = (logp - moved).float(), torch.randn(8, generator=g)
    ref, w = (logp + 0.3).float(), torch.rand(8, generator=g)
    _, _, grad = m.policy_loss(logits.cuda(), tokens.cuda(), old.cuda(), adv.cuda(),
                               ref_logprobs=ref.cuda(), weights=w.cuda(), temperature=0.8, kl_coef=0.2)

    def total(l):
        lp = tc.logprobs(l, tokens, 0.8)[0]
        return float((tc.policy(lp, tokens, 60, old, adv, ref, 0.2, 0.2, 0.2)[0] * w.double()).sum())
    h = 1e-5
    for _ in range(4):
        way = torch.randn(8, 60, generator=g, dtype=torch.float64)
        diff = (total(logits.double() + h * way) - total(logits.double() - h * way)) / (2 * h)
        terms = grad.cpu().double() * way
        # fp32's rounding of each term, and the differences' h^2
        assert abs(diff - float(terms.sum())) <= (60 * U32 + 1e-6) * float(terms.abs().sum())


def offsets_of(kind, rows, pairs, g):
    cuts = torch.randint(0, rows + 1, (2 * pairs + 1,), generator=g).sort().values
    if kind == "whole":
        cuts[0], cuts[-1] = 0, rows
    elif kind == "empty":
        cuts[:] = rows // 2
    return cuts.to(torch.int32)


@pytest.mark.parametrize("rows,pairs", [(1, 1), (2, 1), (40, 3), (1000, 7), (20000, 1), (5000, 300)])
@pytest.mark.parametrize("kind", ["whole", "inside", "empty"])
@pytest.mark.parametrize("beta,smooth,weighted", [(0.1, 0.0, False), (0.5, 0.1, True), (-2.0, 1.0, True),
                                                  (30.0, 0.2, False)])
def test_preference(rows, pairs, kind, beta, smooth, weighted):
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(rows + pairs)
    logp, ref = -3 * torch.rand(rows, generator=g), -3 * torch.rand(rows, generator=g)
    at = offsets_of(kind, rows, pairs, g)
    w = torch.rand(pairs, generator=g) if weighted else None
    loss, grad = m.preference_loss(logp.cuda(), ref.cuda(), at.cuda(), beta=beta, label_smoothing=smooth,
                                   weights=None if w is None else w.cuda())
    want, want_grad, d = tc.preference(logp, ref, at, w, beta, smooth)
    # d is rounded (and beta, which is fp32): what that moves the loss by, at a
    # slope of at most 1, and 8 roundings of the two softplus' sizes
    lc.bound(loss, want, 3 * U32 * d.abs() + 8 * U32 * (d.abs() + 0.7), torch.float32)
    # the sigmoid moves by at most a fourth of what d does
    each = torch.zeros(rows, dtype=torch.float64)
    for p in range(pairs):
        each[at[2 * p]:at[2 * p + 2]] = abs(beta) * (1.0 if w is None else float(w[p])) * (
            float(d[p].abs()) * U32 + 8 * U32)
    lc.bound(grad, want_grad, each, torch.float32)
    out = torch.ones(rows, dtype=torch.bool)
    out[at[0]:at[-1]] = False
    assert (grad.cpu()[out] == 0).all()


def test_preference_offsets_outside():
    """Offsets outside the rows count as the nearest inside, falling ones as empty
    sequences: nothing outside is read or written."""
    import selective_state_space_52_amd as m
    g = torch.Generator().manual_seed(0)
    logp, ref = torch.randn(50, generator=g).cuda(), torch.randn(50, generator=g).cuda()
    wild = torch.tensor([-(1 << 31), 20, (1 << 31) - 1], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    for a, b in zip(m.preference_loss(logp, ref, wild), m.preference_loss(logp, ref, tame)):
        assert torch.equal(a, b)
    falling = torch.tensor([40, 30, 10], dtype=torch.int32, device="cuda")
    loss, grad = m.preference_loss(logp, ref, falling)
    assert abs(float(loss[0]) - 0.6931471805599453) < 1e-6 and (grad == 0).all()


def test_preference_chain_against_differences():
    """The three calls of a preference step against differences of the 64-bit loss
    by the logits."""
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(30, 50, "f32", seed=8)
    ref = tc.logprobs(logits, tokens, 1.0)[0].float() + 0.2 * torch.randn(30, generator=g)
    at = torch.tensor([2, 9, 15, 15, 28], dtype=torch.int32)
    w = torch.tensor([0.4, 1.1])
    logp, stats = m.token_logprobs_fwd(logits.cuda(), tokens.cuda())
    _, d = m.preference_loss(logp, ref.cuda(), at.cuda(), weights=w.cuda(), beta=0.7, label_smoothing=0.1)
    grad = m.token_logprobs_bwd(logits.cuda(), tokens.cuda(), stats, d).cpu().double()

    def total(l):
        lp = tc.logprobs(l, tokens, 1.0)[0]
        return float((tc.preference(lp, ref, at, None, 0.7, 0.1)[0] * w.double()).sum())
    h = 1e-5
    for _ in range(4):
        way = torch.randn(30, 50, generator=g, dtype=torch.float64)
        diff = (total(logits.double() + h * way) - total(logits.double() - h * way)) / (2 * h)
        terms = grad * way
        assert abs(diff - float(terms.sum())) <= (200 * U32 + 1e-6) * float(terms.abs().sum())


def test_streams_and_graphs():
    import selective_state_space_52_amd as m
    logits, tokens, g = inputs(20, 5003, "bf16", seed=9)
    ld, td = logits.cuda(), tokens.cuda()
    old, adv = torch.randn(20, device="cuda"), torch.randn(20, device="cuda")
    at = torch.tensor([0, 8, 20], dtype=torch.int32, device="cuda")

    def step():
        a = m.policy_loss(ld, td, old, adv, ref_logprobs=old, kl_coef=0.1)
        logp, stats = m.token_logprobs_fwd(ld, td)
        loss, d = m.preference_loss(logp, old, at)
        return (*a, logp, loss, d, m.token_logprobs_bwd(ld, td, stats, d))
    base = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(base, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        ld.copy_(torch.randn(20, 5003, generator=g).bfloat16() * 3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_refusals():
    import selective_state_space_52_amd as m
    l, t = torch.zeros(4, 32, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    f, at = torch.zeros(4, device="cuda"), torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    s = torch.zeros(4, 2, device="cuda")
    for call in (lambda: m.token_logprobs_fwd(l.half(), t), lambda: m.token_logprobs_fwd(l, t[:3]),
                 lambda: m.token_logprobs_fwd(l, t.int()), lambda: m.token_logprobs_fwd(l.t(), t),
                 lambda: m.token_logprobs_bwd(l, t, s[:, 0], f), lambda: m.token_logprobs_bwd(l, t, s, f[:3]),
                 lambda: m.token_logprobs_bwd(l, t, s, f, out=l.bfloat16()),
                 lambda: m.policy_loss(l, t, f, f.double()), lambda: m.policy_loss(l, t, f, f, weights=f[:2]),
                 lambda: m.policy_loss(l, t, f, f, want_grad=False, out=l),
                 lambda: m.policy_loss(l, t, f, f, ref_logprobs=f.cpu()),
                 lambda: m.preference_loss(f, f, at.long()), lambda: m.preference_loss(f, f, at[:2]),
                 lambda: m.preference_loss(f, f[:3], at), lambda: m.preference_loss(f, f, at, weights=f)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: m.token_logprobs_fwd(l, t, temperature=0.0),
                 lambda: m.policy_loss(l, t, f, f, clip_low=-0.1),
                 lambda: m.preference_loss(f, f, at, label_smoothing=2.0),
                 lambda: m.token_logprobs_fwd(l[:0], t[:0])):
        with pytest.raises(m.MssmError):
            call()
