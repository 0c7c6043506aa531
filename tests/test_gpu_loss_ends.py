"""The losses where a probability is zero, a ratio or a weight at its type's ends."""
import pytest
import torch

from tests import layer_common as lc
from tests import train_common as tc

pytestmark = pytest.mark.gpu
U32 = lc.U32


@pytest.mark.parametrize("smooth", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("beta", [0.1, -0.1])
def test_preference_of_impossible_answers(smooth, beta):
    """A masked token's log-probability is -infinity, so a pair's difference may be
    infinite: -log sigmoid(+infinity) is 0, of -infinity infinity, and the slope is
    that of the limit."""
    import selective_state_space_52_amd as m
    inf = float("inf")
    logp = torch.tensor([-1.0, -inf, -2.0, -1.5, -inf, -0.5, -1.0, -1.0])
    ref = torch.full((8,), -1.25)
    at = torch.tensor([0, 1, 3, 4, 4, 5, 6, 7, 8], dtype=torch.int32)
    d = torch.tensor([inf, -0.25, -inf, 0.0], dtype=torch.float64) * beta
    loss, grad = m.preference_loss(logp.cuda(), ref.cuda(), at.cuda(), beta=beta, label_smoothing=smooth)
    softplus = lambda x: torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731
    want = torch.zeros(4, dtype=torch.float64)
    if smooth < 1:
        want += (1 - smooth) * softplus(-d)
    if smooth > 0:
        want += smooth * softplus(d)
    # d, beta, the smoothing and its difference from 1, two softplus of 4 roundings
    lc.bound(loss, want, 16 * U32 * (want.nan_to_num(posinf=0.0) + 1), torch.float32)
    slope = (smooth - 1 / (1 + torch.exp(d))) * beta
    sides = torch.stack((slope, -slope), 1).flatten()
    sizes = (at[1:] - at[:-1]).tolist()
    lc.bound(grad, torch.cat([s.expand(n) for s, n in zip(sides, sizes)]), 16 * U32 * abs(beta), torch.float32)


@pytest.mark.parametrize("vocab", [40, 70003])
def test_policy_with_a_token_of_probability_zero(vocab):
    """A ratio of 0, clipped or not; the KL estimate of a token that only the
    reference would take is infinite, of one that only the policy would take too."""
    import selective_state_space_52_amd as m
    inf = float("inf")
    g = torch.Generator().manual_seed(vocab)
    logits = torch.randn(5, vocab, generator=g)
    tokens = torch.full((5,), 7)
    logits[:3, 7] = -inf
    old, adv = torch.full((5,), -2.0), torch.tensor([1.5, -2.0, 1.5, 0.5, 0.5])
    logp = tc.logprobs(logits, tokens, 1.0)[0]
    old[3:] = logp[3:].float()                        # ratios of 1
    args = [x.cuda() for x in (logits, tokens, old, adv)]
    loss, got, grad = m.policy_loss(*args)
    assert (got[:3] == -inf).all() and (grad[:3] == 0).all()
    lc.bound(loss[:3], torch.tensor([0.0, 1.6, 0.0]), 4 * U32, torch.float32)    # -A times 0, 0.8
    ref = torch.tensor([-1.0, -1.0, -inf, -inf, -1.0])
    loss, _, _ = m.policy_loss(*args, ref_logprobs=ref.cuda(), kl_coef=0.1)
    assert (loss[:2] == inf).all() and float(loss[3]) == inf and torch.isfinite(loss[4])
    assert torch.isnan(loss[2])                       # -infinity less -infinity is no number


@pytest.mark.parametrize("vocab", [40, 70003])
def test_policy_with_ratios_past_fp32(vocab):
    """exp of more than 88 is infinite: times an advantage of 0 it is 0, and clipped
    where the advantage is positive."""
    import selective_state_space_52_amd as m
    inf = float("inf")
    g = torch.Generator().manual_seed(vocab)
    logits, tokens = torch.randn(5, vocab, generator=g), torch.full((5,), 7)
    adv = torch.tensor([0.0, -0.0, 2.0, -2.0, 0.0])
    old = torch.full((5,), -200.0)
    old[4] = float("nan")
    loss, _, grad = m.policy_loss(*(x.cuda() for x in (logits, tokens, old, adv)))
    assert (loss[:2] == 0).all() and (grad[:3] == 0).all()
    lc.bound(loss[2:3], torch.tensor([-2.4]), 8 * U32, torch.float32)
    assert float(loss[3]) == inf and torch.isnan(loss[4])


@pytest.mark.parametrize("vocab,io", [(70002, "bf16"), (131072, "bf16"), (70001, "f32"), (50304, "bf16"),
                                      (50257, "f32"), (12000, "bf16")])
def test_rows_alone_and_among_many(vocab, io):
    """A row's log-probability has the same bits in a call of many rows and in one of a
    few, so samples that were scored in one call train in smaller ones with ratios of
    exactly 1; with and without the gradient."""
    import selective_state_space_52_amd as m
    rows = 1024
    g = torch.Generator(device="cuda").manual_seed(vocab)
    logits = torch.randn(rows, vocab, generator=g, device="cuda").to(lc.IO[io])
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logp, stats = m.token_logprobs_fwd(logits, tokens)
    adv = torch.ones(rows, device="cuda")
    for n in (1, 6, 130):
        for at in (0, rows - n):
            part = slice(at, at + n)
            few, few_stats = m.token_logprobs_fwd(logits[part], tokens[part])
            assert torch.equal(few, logp[part]) and torch.equal(few_stats, stats[part])
            loss, again, _ = m.policy_loss(logits[part], tokens[part], logp[part], adv[part])
            assert torch.equal(again, few) and (loss == -1).all()
