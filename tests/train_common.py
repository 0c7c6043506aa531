"""64-bit references of the ends of a training step, and the tolerances of
their tests (U32 and U16 as in layer_common)."""
import math

import torch

from tests.layer_common import U32

M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def embedding(tokens, table, scale):
    live = (tokens >= 0) & (tokens < table.shape[0])
    rows = table.double()[torch.where(live, tokens, 0)] * scale
    return torch.where(live[:, None], rows, 0.0)


def embedding_bwd(tokens, dout, vocab, scale):
    """The gradient, and the sums of the absolute values of its terms times the
    number of terms (what a sum in fp32 is off by, in U32)."""
    total = torch.zeros(vocab, dout.shape[1], dtype=torch.float64)
    size, count = torch.zeros_like(total), torch.zeros(vocab)
    for i, t in enumerate(tokens.tolist()):
        if 0 <= t < vocab:
            total[t] += dout[i].double()
            size[t] += dout[i].double().abs()
            count[t] += 1
    return total * scale, size * abs(scale) * (count[:, None] + 4)


def logprobs(logits, tokens, temperature):
    """Returns (logp, largest logit, log of the sum, softmax) in 64 bits."""
    l = logits.double()
    top = l.amax(1)
    z = (l - top[:, None]) / temperature
    log_sum = torch.log(torch.exp(z).sum(1))
    logp, none = torch.zeros(l.shape[0], dtype=torch.float64), (tokens < 0) | (tokens >= l.shape[1])
    for i, t in enumerate(tokens.tolist()):
        if not none[i]:
            logp[i] = z[i, t] - log_sum[i]
    return logp, top, log_sum, torch.exp(z - log_sum[:, None])


def logprob_slack(logits, tokens, temperature):
    """Absolute errors of logp, of the log of the sum and, relative to them, of
    the probabilities, in fp32.  An exponent (l - top) / T is rounded by its
    difference, three times in its factor log2(e) / T and in their product: 5 U32
    of it, and the hardware exp2 adds 4 U32; a term of the sum is off by that
    much of itself, so the sum by the mean of it under the softmax.  A thread
    adds V / 1024 terms or fewer, rescales (8 U32 a time, at most) its sum every
    8th of them, and 22 joins follow.  The log and the token's own z add 4 U32
    of their sizes."""
    l, v = logits.double(), logits.shape[1]
    z = torch.nan_to_num((l - l.amax(1)[:, None]) / temperature, nan=0.0, neginf=0.0).abs()
    _, _, log_sum, p = logprobs(logits, tokens, temperature)
    mean = (torch.nan_to_num(p) * z).sum(1)
    of_sum = U32 * (5 * mean + 4 + (v / 1024 + 1) * 2 + 22 * 9) + 4 * U32 * log_sum.abs()
    own = z[torch.arange(len(tokens)), tokens.clamp(0, v - 1)]
    return of_sum + 5 * U32 * (own + 1), of_sum, U32 * (6 * z + 8) + of_sum[:, None]


def softmax_slope(p, tokens, factor):
    """factor * ([j = token] - p), rows without a factor zero."""
    d = -factor[:, None] * p
    for i, t in enumerate(tokens.tolist()):
        if 0 <= t < p.shape[1]:
            d[i, t] += factor[i]
        else:
            d[i] = 0.0
        if factor[i] == 0:
            d[i] = 0.0
    return d


def policy(logp, tokens, vocab, old, adv, ref, low, high, kl):
    """(loss, d loss / d logp) of each row, in 64 bits."""
    live = (tokens >= 0) & (tokens < vocab)
    ratio = torch.exp(logp - old.double())
    a = adv.double()
    free, held = ratio * a, ratio.clamp(1 - low, 1 + high) * a
    loss = -torch.minimum(free, held)
    slope = torch.where(free <= held, -free, 0.0)
    if ref is not None:
        x = ref.double() - logp
        loss = loss + kl * (torch.expm1(x) - x)
        slope = slope - kl * torch.expm1(x)
    return torch.where(live, loss, 0.0), torch.where(live, slope, 0.0)


def preference(logp, ref, offsets, weights, beta, smooth):
    """(loss, dlogprobs, d) in 64 bits, pair by pair."""
    gap, at = logp.double() - ref.double(), offsets.tolist()
    loss, diff, grad = [], [], torch.zeros(len(logp), dtype=torch.float64)
    for p in range(len(at) // 2):
        a, b, c = at[2 * p:2 * p + 3]
        d = beta * float(gap[a:b].sum() - gap[b:c].sum())
        minus = max(-d, 0.0) + math.log1p(math.exp(-abs(d)))       # -log sigmoid(d)
        loss.append((1 - smooth) * minus + smooth * (minus + d))
        against = math.exp(-max(d, 0.0)) / (1 + math.exp(-abs(d))) if d > 0 else 1 / (1 + math.exp(d))
        w = (1.0 if weights is None else float(weights[p])) * beta * (smooth - against)
        grad[a:b], grad[b:c] = w, -w
        diff.append(d)
    return torch.tensor(loss, dtype=torch.float64), grad, torch.tensor(diff, dtype=torch.float64)


def dither(n, seed, step):
    """The fractions for m and v, as integers over 2^24."""
    x = (seed + step) * 0x9E3779B97F4A7C15 & M64
    x = (x ^ x >> 32) * 0x6A09E667F3BCC909 & M64
    x ^= x >> 32
    i = torch.arange(n, dtype=torch.int64)
    return (((x & M32) + i * 0x9E3779B9 & M32) >> 8), (((x >> 32) + i * 0x6A09E667 & M32) >> 8)


def values8(q, scales):
    return q.double() * scales.double().repeat_interleave(128)


def adamw(param, grad, m, v, step, lr, b1, b2, eps, decay, grad_scale):
    """(param, m, v) in 64 bits."""
    g = grad.double() * grad_scale
    m, v = b1 * m.double() + (1 - b1) * g, b2 * v.double() + (1 - b2) * g * g
    hat = (m / (1 - b1 ** step)) / (torch.sqrt(v / (1 - b2 ** step)) + eps)
    return param.double() * (1 - lr * decay) - lr * hat, m, v


def check_rounded(q, scales, x, slack, u, positive):
    """q, scales are x in blocks of 128 as the definition has it: the scale the
    block's largest / 448, each value one of the two e4m3 values around x / scale,
    the one that u picks; `slack` is how far x may be off, relative to itself."""
    q, x, u = (t.reshape(-1, 128) for t in (q.double(), x, u))
    most = x.abs().amax(1, keepdim=True)
    most = torch.where(most < 2.0 ** -100, 0.0, most)
    s = scales.double()[:, None]
    assert ((s - most / 448).abs() <= (slack + 2 * U32) * most / 448).all()
    y = torch.where(most > 0, x.abs() / most * 448, 0.0)
    _, e = torch.frexp(y)
    unit = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    place = y / unit + u.double() * 2.0 ** -24
    want = torch.clamp(torch.floor(place) * unit, max=448.0)
    if positive:
        want = torch.where((want == 0) & (x > 0) & (most > 0), 2.0 ** -9, want)
    want = want * torch.sign(x)
    # y is at most 16 units: place is off by 16 (2 slack + 4 U32) and a rounding
    off = 16 * (2 * slack + 6 * U32)
    clear = (place - torch.round(place)).abs() > off
    assert (q == want)[clear].all()
    assert ((q - want).abs() <= 2 * unit)[~clear].all()
