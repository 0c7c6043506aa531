"""Measured cases of the operators of a training step at the model's two ends:
the embedding's rows and their gradient, the log-probabilities of given tokens
with the policy and preference losses on them, and the AdamW step.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, sums along sequences in 64) or, with ``own`` true, through the
library's entry points.  ``exact`` gives the same results in 64 bits.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
FP8_MAX = 448.0        # largest finite e4m3 value
BLOCK = 128            # elements of an 8-bit state that share one scale
SMALLEST = 2.0 ** -100   # a block whose largest value is below this counts as zero
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def listed():
    return [
        # the tokens of a training or prompt batch (4 x 2048) into a 2560-wide stream
        {"name": "embedding, prompt", "op": "embed", "rows": 8192, "vocab": 50304, "dim": 2560,
         "table": "bf16", "io": "bf16", "scale": 1.0},
        # one token of each of 16 sequences, table in fp32: latency
        {"name": "embedding, 16 tokens", "op": "embed", "rows": 16, "vocab": 50257, "dim": 768,
         "table": "f32", "io": "bf16", "scale": 27.7},
        # the gradient of that batch's table, tokens as unevenly spread as a text's
        {"name": "embedding backward", "op": "embed_bwd", "rows": 8192, "vocab": 50304, "dim": 2560,
         "io": "bf16", "grad": "f32", "scale": 1.0, "add": False, "skew": 1.0},
        # a ragged batch added to the gradient that the output projection, which
        # shares the table, has left there
        {"name": "embedding backward, tied", "op": "embed_bwd", "rows": 1777, "vocab": 50257,
         "dim": 769, "io": "f32", "grad": "f32", "scale": 0.5, "add": True, "skew": 1.0},
        # sampled answers of a policy, a fourth of the rows being their prompts
        {"name": "policy loss, 4096 rows", "op": "policy", "rows": 4096, "vocab": 50304,
         "io": "bf16", "temperature": 1.0, "kl": 0.05, "pad": 0, "skip": 0.25},
        # a few tokens, fp32 logits in padded rows: latency
        {"name": "policy loss, 7 rows", "op": "policy", "rows": 7, "vocab": 50257, "io": "f32",
         "temperature": 0.8, "kl": 0.02, "pad": 47, "skip": 0.0},
        # a vocabulary of many languages, at an odd size; no reference policy
        {"name": "policy loss, long rows", "op": "policy", "rows": 1000, "vocab": 200003,
         "io": "bf16", "temperature": 1.0, "kl": 0.0, "pad": 0, "skip": 0.1},
        # 16 pairs of answers packed one after another
        {"name": "preference, 16 pairs", "op": "preference", "rows": 8192, "vocab": 50304,
         "pairs": 16, "io": "bf16", "beta": 0.1, "smooth": 0.0, "skip": 0.4},
        # a few short answers, fp32 logits at an odd vocabulary
        {"name": "preference, 3 pairs", "op": "preference", "rows": 301, "vocab": 32001,
         "pairs": 3, "io": "f32", "beta": 0.2, "smooth": 0.1, "skip": 0.2},
        # every tensor of a 24-layer 768-wide Mamba-2 model, states in fp32, a bf16
        # copy of the weights for the next forward pass
        {"name": "adamw, 24 layers", "op": "adamw", "width": 768, "layers": 24, "vocab": 50304,
         "bits": 32, "grad": "bf16", "copy": True},
        # two 2560-wide layers and the table, states in 8 bits
        {"name": "adamw, 8 bits", "op": "adamw", "width": 2560, "layers": 2, "vocab": 50304,
         "bits": 8, "grad": "bf16", "copy": True},
        # a small model's tensors, fp32 gradients, no copy: latency
        {"name": "adamw, small", "op": "adamw", "width": 96, "layers": 2, "vocab": 257,
         "bits": 8, "grad": "f32", "copy": False},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed", "embed_bwd", "policy", "preference", "adamw"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "embed":
        return {"op": op, "rows": size(1, 8192), "vocab": size(256, 50304), "dim": size(64, 2560),
                "table": rng.choice(["bf16", "f32"]), "io": io, "scale": rng.choice([1.0, 16.0])}
    if op == "embed_bwd":
        return {"op": op, "rows": size(1, 8192), "vocab": size(256, 50304), "dim": size(64, 2560),
                "io": io, "grad": rng.choice(["f32", "f32", "bf16"]),
                "scale": rng.choice([1.0, 16.0]), "add": rng.random() < 0.4,
                "skew": rng.choice([0.0, 1.0, 1.5])}
    if op == "policy":
        return {"op": op, "rows": size(1, 2048), "vocab": size(1000, 100000), "io": io,
                "temperature": rng.choice([1.0, 0.7]), "kl": rng.choice([0.0, 0.05]),
                "pad": rng.choice([0, 7, 64]), "skip": rng.choice([0.0, 0.3])}
    if op == "preference":
        pairs = size(1, 16)
        return {"op": op, "rows": size(4 * pairs, 2048), "vocab": size(1000, 100000),
                "pairs": pairs, "io": io, "beta": rng.choice([0.1, 0.3]),
                "smooth": rng.choice([0.0, 0.1]), "skip": rng.choice([0.0, 0.4])}
    return {"op": op, "width": 32 * size(2, 60), "layers": size(1, 4), "vocab": size(256, 20000),
            "bits": rng.choice([8, 32]), "grad": rng.choice(["bf16", "f32"]),
            "copy": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _shapes(case):
    """The tensors of a Mamba-2 model of this width (heads of 64 channels, an
    expansion of 2, one group of 128 states, convolution of width 4), the
    matrices first in each layer."""
    width, heads = case["width"], case["width"] // 32
    inner = 2 * width
    channels = inner + 256
    layer = [(inner + channels + heads, width), (width, inner), (channels, 4), (channels,),
             (heads,), (heads,), (heads,), (inner,), (width,)]
    return [(case["vocab"], width)] + layer * case["layers"] + [(width,)]


def _sizes(case):
    return [math.prod(s) for s in _shapes(case)]


def _live(case):
    return case["rows"] - int(case["rows"] * case["skip"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 % (1 << 62))

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    op = case["op"]
    s = {"case": case}
    if op in ("embed", "embed_bwd"):
        rows, vocab, dim = case["rows"], case["vocab"], case["dim"]
        # tokens whose frequency falls as rank ** -skew, ranks spread over the table
        weight = (1.0 + torch.arange(vocab, device="cuda")).pow(-case.get("skew", 1.0))
        rank = torch.multinomial(weight, rows, replacement=True, generator=g)
        s["tokens"] = torch.randperm(vocab, generator=g, device="cuda")[rank]
        if op == "embed":
            s["table"] = randn(vocab, dim, dtype=DTYPES[case["table"]], scale=0.02)
        else:
            s["dout"] = randn(rows, dim, dtype=DTYPES[case["io"]], scale=1e-2)
            s["dtable"] = randn(vocab, dim, dtype=DTYPES[case["grad"]], scale=1e-2) if case["add"] else None
        return s
    if op in ("policy", "preference"):
        rows, vocab, pad = case["rows"], case["vocab"], case.get("pad", 0)
        logits = randn(rows, vocab + pad, scale=2.0)
        # a few tokens stand out, as a trained model's do, and are mostly the ones taken
        hot = torch.randint(0, vocab, (rows, 12), generator=g, device="cuda")
        logits.scatter_add_(1, hot, 5.0 + 5.0 * rand(rows, 12))
        logits = logits.to(DTYPES[case["io"]])[:, :vocab]
        tokens = torch.where(rand(rows) < 0.9, hot[:, 0], torch.randint(0, vocab, (rows,), generator=g,
                                                                        device="cuda"))
        temperature = case.get("temperature", 1.0)
        z = logits.double().div_(temperature)
        logp = (z.gather(1, tokens[:, None]).squeeze(1) - torch.logsumexp(z, 1)).float()
        del z
        # rows of the prompt have no token of their own
        skip = torch.randperm(rows, generator=g, device="cuda")[:rows - _live(case)]
        tokens[skip] = -1
        s["logits"], s["tokens"] = logits, tokens
        if op == "policy":
            # the policy has moved a little since it sampled: ratios around 1, some
            # of them past the clip, none within 1e-3 of it
            moved = 0.15 * torch.randn(rows, generator=g, device="cuda")
            for edge in (math.log(0.8), math.log(1.2)):
                moved = torch.where((moved - edge).abs() < 1e-3, moved + 3e-3, moved)
            s["old"] = logp - moved
            s["advantages"] = randn(rows)
            s["weights"] = (0.5 + rand(rows)) / rows
            s["ref"] = logp + 0.2 * randn(rows) if case["kl"] else None
        else:
            s["ref"] = logp + 0.1 * randn(rows)
            s["ref"][skip] = 0.0
            ends = torch.randperm(rows - 1, generator=g, device="cuda")[:2 * case["pairs"] - 1] + 1
            s["offsets"] = torch.cat((ends.new_zeros(1), ends.sort().values,
                                      ends.new_full((1,), rows))).to(torch.int32)
            s["weights"] = (0.5 + rand(case["pairs"])) / case["pairs"]
        return s
    shapes, sizes = _shapes(case), _sizes(case)
    total, padded = sum(sizes), [-(-n // BLOCK) * BLOCK for n in sizes]

    def views(flat):
        return [v.view(shape) for v, shape in zip(flat.split(sizes), shapes)]

    s["flat"] = randn(total, scale=0.02)
    s["params"] = views(s["flat"])
    s["grads"] = views((randn(total) * torch.exp(randn(total))).mul_(1e-3).to(DTYPES[case["grad"]]))
    s["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
    s["copies"] = views(s["copy"]) if case["copy"] else None
    s["decay"] = [0.1 if len(shape) == 2 and shape[1] != 4 else 0.0 for shape in shapes]
    s["grad_scale"] = 0.5 + 0.5 * rand(1)
    s["step"], s["seed"] = 1000, int(seed) & M32
    # where there is an element, its moments; zero between one tensor's end and
    # the next multiple of 128, where the next one's begin
    there = torch.cat([(torch.arange(p, device="cuda") < n) for n, p in zip(sizes, padded)])
    m = torch.where(there, randn(sum(padded), scale=3e-4), 0.0)
    root = torch.where(there, 1e-3 * torch.exp(randn(sum(padded), scale=0.7)), 0.0)
    s["m_scales"] = s["v_scales"] = None
    if case["bits"] == 8:
        half = torch.full_like(m, 0.5)
        s["m"], s["m_scales"] = _to_8_bits(m, half, False)
        s["v"], s["v_scales"] = _to_8_bits(root, half, True)
    else:
        s["m"], s["v"] = m, root.square_()
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits

def _plain_embed(s):
    rows = s["table"][s["tokens"]].float()
    return (rows * s["case"]["scale"]).to(DTYPES[s["case"]["io"]])


def _plain_embed_bwd(s):
    case = s["case"]
    total = torch.zeros(case["vocab"], case["dim"], device="cuda")
    total.index_add_(0, s["tokens"], s["dout"].float())
    total = total * case["scale"]
    if not case["add"]:
        return total.to(DTYPES[case["grad"]])
    s["dtable"].copy_(s["dtable"].float() + total)
    return s["dtable"]


def _plain_logprobs(logits, tokens, temperature):
    """Log-probabilities of the tokens (0 for none) and the rows' normalisers."""
    z = logits.float() / temperature
    top = z.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True))).squeeze(1)
    live = tokens >= 0
    taken = z.gather(1, tokens.clamp(min=0)[:, None]).squeeze(1)
    return torch.where(live, taken - lse, 0.0), lse


def _plain_logits_grad(logits, tokens, lse, factor, temperature):
    """factor * d logprob / d logits, in the logits' type."""
    live = tokens >= 0
    factor = torch.where(live, factor / temperature, 0.0)[:, None]
    d = -factor * torch.exp(logits.float() / temperature - lse[:, None])
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], factor)
    return d.to(logits.dtype)


def _plain_policy(s):
    case = s["case"]
    logp, lse = _plain_logprobs(s["logits"], s["tokens"], case["temperature"])
    ratio, adv = torch.exp(logp - s["old"]), s["advantages"]
    free, held = ratio * adv, ratio.clamp(0.8, 1.2) * adv
    loss = -torch.minimum(free, held)
    slope = torch.where(free <= held, -free, 0.0)
    if s["ref"] is not None:
        x = s["ref"] - logp
        loss = loss + case["kl"] * (torch.expm1(x) - x)
        slope = slope - case["kl"] * torch.expm1(x)
    loss = torch.where(s["tokens"] >= 0, loss, 0.0)
    return loss, logp, _plain_logits_grad(s["logits"], s["tokens"], lse, slope * s["weights"],
                                          case["temperature"])


def _plain_preference(s):
    case = s["case"]
    logp, lse = _plain_logprobs(s["logits"], s["tokens"], 1.0)
    at = s["offsets"].long()
    ahead = torch.nn.functional.pad(torch.cumsum((logp - s["ref"]).double(), 0), (1, 0))
    of_sequence = ahead[at[1:]] - ahead[at[:-1]]
    d = case["beta"] * (of_sequence[0::2] - of_sequence[1::2])
    softplus = lambda x: torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731
    loss = (1.0 - case["smooth"]) * softplus(-d) + case["smooth"] * softplus(d)
    slope = (1.0 / (1.0 + torch.exp(-d)) - (1.0 - case["smooth"])) * case["beta"] * s["weights"]
    sign = torch.stack((slope, -slope), 1).flatten().float()
    row = torch.arange(case["rows"], device="cuda")
    factor = sign[torch.searchsorted(at[1:], row, right=True)]
    return loss.float(), logp, factor, _plain_logits_grad(s["logits"], s["tokens"], lse, factor, 1.0)


def _dither(n, shift, stride):
    """n fractions in [0, 1): shift + i * stride modulo 2^32, its upper 24 bits."""
    i = torch.arange(n, device="cuda", dtype=torch.int64)
    return (((i * stride + shift) & M32) >> 8).float() * 2.0 ** -24


def _shifts(seed, step):
    """The two words that shift a step's dither."""
    x = (seed + step) * 0x9E3779B97F4A7C15 & M64
    x = (x ^ x >> 32) * 0x6A09E667F3BCC909 & M64
    x ^= x >> 32
    return x & M32, x >> 32


def _to_8_bits(x, u, positive):
    """x (whole blocks) as e4m3 with the scale max / 448 a block, each value to
    the one above or below it as u in [0, 1) says; where all are positive, none
    of them to zero.  Returns the values and the scales."""
    x = x.view(-1, BLOCK)
    most = x.abs().amax(1, keepdim=True)
    most = torch.where(most < SMALLEST, 0.0, most)
    y = x * torch.where(most > 0, FP8_MAX / most, 0.0)
    exponent = (y.abs().view(torch.int32) >> 23).clamp(min=121)        # biased: 2^-6 and up
    unit = ((exponent - 3) << 23).view(torch.float32)                   # 3 mantissa bits
    size = (torch.floor(y.abs() / unit + u.view(-1, BLOCK)) * unit).clamp(max=FP8_MAX)
    if positive:
        size = torch.where((x > 0) & (most > 0), size.clamp(min=2.0 ** -9), size)
    return torch.copysign(size, y).to(F8).flatten(), (most / FP8_MAX).flatten()


def _from_8_bits(q, scales):
    return (q.float().view(-1, BLOCK) * scales[:, None]).flatten()


LR, BETA1, BETA2, EPS = 3e-4, 0.9, 0.95, 1e-8


def _plain_adamw_one(s, param, grad, decay, at, copy):
    """One tensor's step, its moments from element `at` of theirs."""
    n = param.numel()
    padded = -(-n // BLOCK) * BLOCK
    part, blocks = slice(at, at + padded), slice(at // BLOCK, (at + padded) // BLOCK)
    eight = s["case"]["bits"] == 8
    g = torch.nn.functional.pad(grad.flatten().float() * s["grad_scale"], (0, padded - n))
    m = _from_8_bits(s["m"][part], s["m_scales"][blocks]) if eight else s["m"][part]
    v = _from_8_bits(s["v"][part], s["v_scales"][blocks]).square() if eight else s["v"][part]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    root = torch.sqrt(v)
    if eight:
        low, high = _shifts(s["seed"], s["step"])
        s["m"][part], s["m_scales"][blocks] = _to_8_bits(m, _dither(padded, low, 0x9E3779B9), False)
        s["v"][part], s["v_scales"][blocks] = _to_8_bits(root, _dither(padded, high, 0x6A09E667), True)
    else:
        s["m"][part], s["v"][part] = m, v
    c1, c2 = 1.0 - BETA1 ** s["step"], math.sqrt(1.0 - BETA2 ** s["step"])
    update = (m / c1 / (root / c2 + EPS))[:n].view(param.shape)
    param.copy_(param * (1.0 - LR * decay) - LR * update)
    if copy is not None:
        copy.copy_(param)


def _adamw_outputs(s):
    return {k: s[k] for k in ("flat", "copy", "m", "v", "m_scales", "v_scales") if s[k] is not None}


def _plain_adamw(s):
    at = 0
    copies = s["copies"] or [None] * len(s["params"])
    for param, grad, decay, copy in zip(s["params"], s["grads"], s["decay"], copies):
        _plain_adamw_one(s, param, grad, decay, at, copy)
        at += -(-param.numel() // BLOCK) * BLOCK
    return _adamw_outputs(s)


_PLAIN = {"embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "policy": _plain_policy,
          "preference": _plain_preference, "adamw": _plain_adamw}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import selective_state_space_52_amd as mssm
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return mssm.embedding_fwd(s["tokens"], s["table"], scale=case["scale"],
                                  out_dtype=DTYPES[case["io"]])
    if op == "embed_bwd" and case["add"]:
        return mssm.embedding_bwd(s["tokens"], s["dout"], case["vocab"], scale=case["scale"],
                                  add_to=s["dtable"])
    if op == "embed_bwd":
        return mssm.embedding_bwd(s["tokens"], s["dout"], case["vocab"], scale=case["scale"],
                                  out_dtype=DTYPES[case["grad"]])
    if op == "policy":
        return mssm.policy_loss(s["logits"], s["tokens"], s["old"], s["advantages"],
                                ref_logprobs=s["ref"], weights=s["weights"],
                                temperature=case["temperature"], clip_low=0.2, clip_high=0.2,
                                kl_coef=case["kl"])
    if op == "preference":
        logp, lse = mssm.token_logprobs_fwd(s["logits"], s["tokens"])
        loss, factor = mssm.preference_loss(logp, s["ref"], s["offsets"], weights=s["weights"],
                                            beta=case["beta"], label_smoothing=case["smooth"])
        return loss, logp, factor, mssm.token_logprobs_bwd(s["logits"], s["tokens"], lse, factor)
    mssm.adamw_step(s["params"], s["grads"], s["m"], s["v"], step=s["step"], lr=LR,
                    betas=(BETA1, BETA2), eps=EPS, weight_decay=s["decay"],
                    m_scales=s["m_scales"], v_scales=s["v_scales"], copies=s["copies"],
                    grad_scale=s["grad_scale"], seed=s["seed"])
    return _adamw_outputs(s)


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- floors

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "embed":
        e = case["rows"] * case["dim"]
        return {"bytes": e * (size[case["table"]] + size[case["io"]]) + 8 * case["rows"], "flops": e}
    if op == "embed_bwd":
        rows, vocab, dim = case["rows"], case["vocab"], case["dim"]
        # added to: only the rows that tokens name, each read and written (as
        # many as the expected number of different tokens of an even spread, at most)
        named = vocab * -math.expm1(rows * math.log1p(-1.0 / vocab)) if case["add"] else vocab
        if case["add"] and case["skew"]:
            named *= 0.5
        return {"bytes": rows * (dim * size[case["io"]] + 8)
                + named * dim * size[case["grad"]] * (2 if case["add"] else 1), "flops": rows * dim}
    if op in ("policy", "preference"):
        # the rows that have a token are read (twice where the loss joins rows before
        # their gradient is known) and every row's gradient is written
        reads = 2 if op == "preference" else 1
        e = (_live(case) * reads + case["rows"]) * case["vocab"]
        return {"bytes": e * size[case["io"]] + 40 * case["rows"],
                "flops": 8 * _live(case) * case["vocab"]}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (8 + size[case["grad"]] + state + (2 if case["copy"] else 0)),
            "flops": 16 * n}


# ---------------------------------------------------------------- the same in 64 bits

def _exact_losses(s):
    """Row by row of the definitions: softmax in 64 bits, the loss's derivative
    by the chosen token's log-probability, and through the softmax."""
    case = s["case"]
    t = case.get("temperature", 1.0)
    has = s["tokens"] >= 0
    index = torch.where(has, s["tokens"], 0).unsqueeze(1)
    logp_all = torch.log_softmax(s["logits"].double() / t, 1)
    logp = torch.where(has, torch.gather(logp_all, 1, index).squeeze(1), 0.0)
    if case["op"] == "policy":
        delta = logp - s["old"].double()
        adv = s["advantages"].double()
        clipped = ((adv > 0) & (delta > math.log(1.2))) | ((adv < 0) & (delta < math.log(0.8)))
        bounded = torch.where(clipped, torch.where(adv > 0, 1.2, 0.8), torch.exp(delta))
        loss = -adv * bounded
        slope = torch.where(clipped, 0.0, -adv * torch.exp(delta))
        if s["ref"] is not None:
            x = s["ref"].double() - logp
            loss = loss + case["kl"] * (torch.exp(x) - 1.0 - x)
            slope = slope + case["kl"] * (1.0 - torch.exp(x))
        loss = torch.where(has, loss, 0.0)
        factor = slope * s["weights"].double()
        first = (loss, logp)
    else:
        gap = (logp - s["ref"].double()).cpu()
        ends = s["offsets"].tolist()
        factor = torch.zeros(case["rows"], dtype=torch.float64)
        loss = []
        for p in range(case["pairs"]):
            a, b, c = ends[2 * p], ends[2 * p + 1], ends[2 * p + 2]
            d = case["beta"] * float(gap[a:b].sum() - gap[b:c].sum())
            chosen = 1.0 / (1.0 + math.exp(-d))
            loss.append(-(1.0 - case["smooth"]) * math.log(chosen)
                        - case["smooth"] * math.log(1.0 - chosen))
            w = float(s["weights"][p]) * case["beta"] * (chosen - 1.0 + case["smooth"])
            factor[a:b], factor[b:c] = w, -w
        factor = factor.cuda()
        first = (torch.tensor(loss, dtype=torch.float64, device="cuda"), logp, factor)
    factor = torch.where(has, factor, 0.0) / t
    grad = torch.exp(logp_all).mul_(-factor.unsqueeze(1))
    grad[torch.arange(case["rows"], device="cuda"), index.squeeze(1)] += factor
    return first + (grad,)


def _exact_e4m3(x, u, positive):
    """As the definition reads: of the two e4m3 values around x * 448 / max the
    upper one where the distance from the lower one and u make a whole step."""
    blocks = x.reshape(-1, BLOCK)
    most = blocks.abs().max(1, keepdim=True).values
    most[most < SMALLEST] = 0.0
    y = torch.where(most > 0, blocks.abs() / most * FP8_MAX, 0.0)
    _, exponent = torch.frexp(y)
    unit = torch.exp2((exponent - 1).clamp(min=-6).double() - 3.0)
    lower = torch.floor(y / unit)
    up = (y / unit - lower) + u.reshape(-1, BLOCK) >= 1.0
    value = torch.clamp((lower + up) * unit, max=FP8_MAX)
    if positive:
        value = torch.where((value == 0) & (blocks > 0) & (most > 0), 2.0 ** -9, value)
    return (value * torch.sign(blocks)).reshape(-1), (most / FP8_MAX).reshape(-1)


def _exact_adamw(s):
    case = s["case"]
    eight, sizes = case["bits"] == 8, _sizes(case)
    out = {k: v.double() for k, v in _adamw_outputs(s).items()}
    scale = s["grad_scale"].double()
    x = (s["seed"] + s["step"]) * 0x9E3779B97F4A7C15 % 2 ** 64
    x = (x ^ (x >> 32)) * 0x6A09E667F3BCC909 % 2 ** 64
    x = x ^ (x >> 32)
    start = at = 0
    for n, grad, decay in zip(sizes, s["grads"], s["decay"]):
        whole = (n + BLOCK - 1) // BLOCK * BLOCK
        g = torch.zeros(whole, dtype=torch.float64, device="cuda")
        g[:n] = grad.reshape(-1).double() * scale
        m, v = out["m"][at:at + whole], out["v"][at:at + whole]
        if eight:
            m = m * out["m_scales"][at // BLOCK:(at + whole) // BLOCK].repeat_interleave(BLOCK)
            v = (v * out["v_scales"][at // BLOCK:(at + whole) // BLOCK].repeat_interleave(BLOCK)) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        if eight:
            i = torch.arange(whole, device="cuda")
            for name, value, word, stride in (("m", m, x % 2 ** 32, 0x9E3779B9),
                                              ("v", v.sqrt(), x // 2 ** 32, 0x6A09E667)):
                u = torch.div((word + i * stride) % 2 ** 32, 256, rounding_mode="floor").double() / 2 ** 24
                q, scales = _exact_e4m3(value, u, name == "v")
                out[name][at:at + whole] = q
                out[name + "_scales"][at // BLOCK:(at + whole) // BLOCK] = scales
        else:
            out["m"][at:at + whole], out["v"][at:at + whole] = m, v
        mhat = m[:n] / (1 - BETA1 ** s["step"])
        vhat = v[:n] / (1 - BETA2 ** s["step"])
        p = out["flat"][start:start + n]
        p += -LR * decay * p - LR * mhat / (torch.sqrt(vhat) + EPS)
        start, at = start + n, at + whole
    if "copy" in out:
        out["copy"] = out["flat"].clone()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        return torch.nn.functional.embedding(s["tokens"], s["table"].double()) * case["scale"]
    if case["op"] == "embed_bwd":
        total = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        total.index_put_((s["tokens"],), s["dout"].double() * case["scale"], accumulate=True)
        return total if s["dtable"] is None else total + s["dtable"].double()
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_losses(s)
