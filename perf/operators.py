"""Measured cases of the layer operators around the scans: the norm that joins
the residual stream, the 8-bit products and their quantiser, the Mamba-2
single-token step, and the choice of the next token.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` true, through the library's entry points.  ``exact``
gives the same results in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128            # columns that share one scale
FP8_MAX = 448.0        # largest finite e4m3 value
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one training or prompt batch (4 x 2048 tokens) of a 2560-wide residual
        # stream kept in fp32, normed into the 8-bit input of the projection
        {"name": "norm to 8 bits, prompt", "op": "norm", "rows": 8192, "dim": 2560, "io": "bf16",
         "res": "f32", "quantize": True},
        # the same for one token of one sequence: latency
        {"name": "norm to 8 bits, 1 token", "op": "norm", "rows": 1, "dim": 2560, "io": "bf16",
         "res": "f32", "quantize": True},
        # odd width and row count, bf16 residual stream, bf16 output
        {"name": "norm, odd width", "op": "norm", "rows": 1777, "dim": 1537, "io": "bf16",
         "res": "bf16", "quantize": False},
        # the norm's training step
        {"name": "norm backward", "op": "norm_bwd", "rows": 8192, "dim": 2560, "io": "bf16",
         "res": "f32"},
        # the input projection of an 80-head Mamba-2 layer (z, x, B, C, dt) over a prompt
        {"name": "product, prompt", "op": "matmul", "m": 8192, "n": 10576, "k": 2560, "out": "bf16"},
        # the same for one token of each of 16 sequences: the weights' bytes
        {"name": "product, 16 tokens", "op": "matmul", "m": 16, "n": 10576, "k": 2560, "out": "bf16"},
        # a 768-wide layer's output projection of a ragged prompt, from bf16 activations
        {"name": "quantise and product, ragged", "op": "linear", "m": 1000, "n": 768, "k": 1536,
         "io": "bf16", "out": "bf16"},
        # the training step of a 768-wide layer's input projection: dX and dW
        {"name": "linear backward", "op": "linear_bwd", "m": 4096, "n": 3352, "k": 768, "io": "bf16"},
        # next tokens of a full serving batch, every request with its own settings
        {"name": "sample, 256 rows", "op": "sample", "rows": 256, "vocab": 50304, "io": "bf16",
         "temperature": 0.9, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "per_row": True, "pad": 64},
        # next token of one sequence
        {"name": "sample, 1 row", "op": "sample", "rows": 1, "vocab": 50257, "io": "f32",
         "temperature": 0.8, "top_k": 50, "top_p": 0.9, "min_p": 0.02, "per_row": False, "pad": 0},
        # one token of each of 256 sequences through an 80-head Mamba-2 layer's
        # convolution and scan, the sequences in slots of a larger cache
        {"name": "step, 256 sequences", "op": "step", "batch": 256, "heads": 80, "groups": 1,
         "n": 128, "io": "bf16", "slots": True},
        # one token of one sequence through a 24-head layer: latency
        {"name": "step, 1 sequence", "op": "step", "batch": 1, "heads": 24, "groups": 1, "n": 128,
         "io": "bf16", "slots": False},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return v + 1 if v == 3072 else v

    op = rng.choice(["norm", "norm", "norm_bwd", "matmul", "matmul", "linear", "linear_bwd",
                     "sample", "sample", "step", "step"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        return {"op": op, "rows": size(1, 8192), "dim": size(64, 2560), "io": io,
                "res": rng.choice(["none", "bf16", "f32"]), "quantize": rng.random() < 0.6}
    if op == "norm_bwd":
        return {"op": op, "rows": size(1, 8192), "dim": size(64, 2560), "io": io,
                "res": rng.choice(["none", "bf16", "f32"])}
    if op in ("matmul", "linear", "linear_bwd"):
        n, k = size(64, 10576), size(64, 5120)
        if rng.random() < 0.7:   # most widths are multiples of 16
            n, k = max(16, n // 16 * 16), max(16, k // 16 * 16)
        n, k = n + 16 * (n == 3072), k + 16 * (k == 3072)
        if op == "matmul":
            return {"op": op, "m": size(1, 4096), "n": n, "k": k, "out": rng.choice(["bf16", "f32"])}
        if op == "linear":
            return {"op": op, "m": size(1, 4096), "n": n, "k": k, "io": io,
                    "out": rng.choice(["bf16", "f32"])}
        return {"op": op, "m": size(64, 2048), "n": n, "k": k, "io": io}
    if op == "sample":
        return {"op": op, "rows": size(1, 256), "vocab": size(1000, 50304), "io": io,
                "temperature": rng.choice([0.0, 0.7, 1.0, 1.3]),
                "top_k": rng.choice([0, 1, size(2, 64), size(64, 1000)]),
                "top_p": rng.choice([1.0, 0.95, 0.8]), "min_p": rng.choice([0.0, 0.05]),
                "per_row": rng.random() < 0.5, "pad": rng.choice([0, 7, 64])}
    n, groups = rng.choice([64, 128]), rng.choice([1, 1, 2])
    heads = groups * size(8, 80) // groups // groups * groups
    if heads * 64 + 2 * groups * n == 3072:
        heads -= groups
    return {"op": op, "batch": size(1, 256), "heads": heads, "groups": groups, "n": n, "io": io,
            "slots": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 % (1 << 62))

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, dim, io = case["rows"], case["dim"], DTYPES[case["io"]]
        res = DTYPES.get(case["res"])
        s = {"case": case, "eps": 1e-5, "weight": 1.0 + randn(dim, scale=0.2)}
        # a residual stream's channels differ in size
        spread = torch.exp(randn(dim, scale=0.7))
        if op == "norm":
            s["x"] = randn(rows, dim).mul_(spread).to(io)
            s["residual"] = None if res is None else (3 * randn(rows, dim) * spread).to(res)
        else:
            s["dout"] = randn(rows, dim, dtype=io, scale=1e-2)
            s["r"] = (3 * randn(rows, dim) * spread).to(io if res is None else res)
            s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + s["eps"])
            s["dresidual"] = None if res is None else randn(rows, dim, dtype=res, scale=1e-2)
        return s
    if op in ("matmul", "linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        s = {"case": case}
        w = randn(n, k, scale=k ** -0.5)
        s["b"], s["b_scales"] = _quantize(w, rows=BLOCK)
        x = randn(m, k) * torch.exp(randn(k, scale=0.7))
        if op == "matmul":
            s["a"], s["a_scales"] = _quantize(x)
        else:
            s["x"] = x.to(DTYPES[case["io"]])
        if op == "linear_bwd":   # the weight's transposed copy, kept beside it for training
            s["wt"], s["wt_scales"] = _quantize(w.t().contiguous(), rows=BLOCK)
            s["dout"] = randn(m, n, dtype=DTYPES[case["io"]], scale=1e-2)
        return s
    if op == "sample":
        rows, vocab, pad = case["rows"], case["vocab"], case["pad"]
        logits = randn(rows, vocab + pad, scale=2.5)
        # a few tokens stand out, as a trained model's do
        hot = torch.randint(0, vocab, (rows, 20), generator=g, device="cuda")
        logits.scatter_add_(1, hot, 4.0 + 4.0 * rand(rows, 20))
        s = {"case": case, "logits": logits.to(DTYPES[case["io"]])[:, :vocab], "noise": rand(rows, vocab)}
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = (
            case["temperature"], case["top_k"], case["top_p"], case["min_p"])
        if case["per_row"]:
            s["temperature"] = case["temperature"] * (0.8 + 0.4 * rand(rows))
            s["top_k"] = torch.ceil(case["top_k"] * (0.5 + 0.5 * rand(rows))).to(torch.int32)
            s["top_p"] = 1.0 - (1.0 - case["top_p"]) * 2.0 * rand(rows)
            s["min_p"] = case["min_p"] * 2.0 * rand(rows)
        return s
    batch, heads, n, groups = case["batch"], case["heads"], case["n"], case["groups"]
    io = DTYPES[case["io"]]
    d, bc = heads * 64, 2 * groups * n
    s = {"case": case}
    cache = batch + (batch + 7) // 8 if case["slots"] else batch
    s["slots"] = None
    if case["slots"]:
        s["slots"] = torch.randperm(cache, generator=g, device="cuda")[:batch].to(torch.int32)
    # z | x, B, C | dt of one projection's output
    proj = randn(batch, 2 * d + bc + heads, dtype=io)
    s["z"], s["xbc"], s["dt"] = proj[:, :d], proj[:, d:2 * d + bc], proj[:, 2 * d + bc:]
    s["state"] = randn(cache, d, n, scale=0.1)
    s["conv_state"] = randn(cache, d + bc, 3, dtype=io)
    s["conv_weight"] = randn(d + bc, 4, scale=0.5)
    s["conv_bias"] = randn(d + bc, scale=0.1)
    s["A"] = -1.0 - 15.0 * rand(heads)
    s["D"] = randn(heads)
    step = torch.exp(rand(heads) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits

def _scale_codes(amax):
    """Biased exponents of the smallest powers of two s with amax / s <= 448."""
    bits = amax.contiguous().view(torch.int32)
    return (((bits + 0x1FFFFF) >> 23) - 8).clamp(0, 254)


def _quantize(x, rows=1):
    """e4m3 values of x and one e8m0 scale for each `rows` x 128 block."""
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - k, 0, mb * rows - m))
    v = v.view(mb, rows, kb, BLOCK)
    code = _scale_codes(v.abs().amax(dim=(1, 3)))
    inverse = ((254 - code) << 23).view(torch.float32)
    q = (v * inverse[:, None, :, None]).view(mb * rows, kb * BLOCK)[:m, :k].to(F8)
    return q.contiguous(), code.to(torch.uint8).view(E8)


def _wide(scales, rows, cols):
    """Scales repeated over their blocks, as 32-bit values."""
    v = scales.float().repeat_interleave(BLOCK, dim=1)[:, :cols]
    return v if v.shape[0] == rows else v.repeat_interleave(BLOCK, dim=0)[:rows]


def _matmul(a, a_scales, b, b_scales, dtype):
    left = a.float() * _wide(a_scales, *a.shape)
    right = b.float() * _wide(b_scales, *b.shape)
    return (left @ right.t()).to(dtype)


def _plain_norm(s):
    case = s["case"]
    r = s["x"].float()
    r = r if s["residual"] is None else r + s["residual"].float()
    rstd = torch.rsqrt(r.square().mean(1, keepdim=True) + s["eps"])
    y = r * rstd * s["weight"]
    stream = None if s["residual"] is None else r.to(s["residual"].dtype)
    if case["quantize"]:
        q, scales = _quantize(y)
        return q, scales, stream
    return y.to(s["x"].dtype), stream


def _plain_norm_bwd(s):
    r, rstd = s["r"].float(), s["rstd"][:, None]
    dy, xhat = s["dout"].float(), r * rstd
    wdy = dy * s["weight"]
    dr = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
    dr = dr if s["dresidual"] is None else dr + s["dresidual"].float()
    stream = None if s["dresidual"] is None else dr.to(s["dresidual"].dtype)
    return dr.to(s["dout"].dtype), stream, (dy * xhat).sum(0)


def _plain_linear_bwd(s):
    dout, x = s["dout"], s["x"]
    dx = _matmul(*_quantize(dout), s["wt"], s["wt_scales"], x.dtype)
    dw = _matmul(*_quantize(dout.t()), *_quantize(x.t()), torch.float32)
    return dx, dw


def _per_row(v, like):
    return v[:, None].float() if isinstance(v, torch.Tensor) else torch.full_like(like, float(v))


def _plain_sample(s):
    t = s["logits"].float()
    rows, vocab = t.shape
    temperature, top_k, top_p, min_p = (_per_row(s[name], t[:, :1]) for name in
                                        ("temperature", "top_k", "top_p", "min_p"))
    sorted_t, order = torch.sort(t, dim=1, descending=True, stable=True)
    greedy = temperature == 0
    scaled = (sorted_t - sorted_t[:, :1]) / torch.where(greedy, 1.0, temperature)
    w = torch.exp(scaled)
    rank = torch.arange(vocab, device=t.device)[None]
    w = torch.where((rank < top_k) | (top_k <= 0), w, 0.0)
    before = torch.cumsum(w, dim=1) - w
    keep = (before < top_p * w.sum(1, keepdim=True)) | (top_p >= 1)
    keep = ((keep & (w >= min_p) & (w > 0)) | (rank == 0)) & ~(greedy & (rank > 0))
    w = torch.where(keep, w, 0.0)
    race = torch.where(keep, w / -torch.log(torch.gather(s["noise"], 1, order)), -1.0)
    # the lowest index among the winners
    best = race == race.amax(1, keepdim=True)
    token = torch.where(best, order, vocab).amin(1)
    won = (best & (order == token[:, None])).float()
    logprob = (torch.where(won > 0, scaled, 0.0)).sum(1) - torch.log(w.sum(1))
    return token, logprob


def _plain_step(s):
    case = s["case"]
    batch, heads, n, groups = case["batch"], case["heads"], case["n"], case["groups"]
    d = heads * 64
    at = slice(None) if s["slots"] is None else s["slots"].long()
    window = torch.cat((s["conv_state"][at], s["xbc"][:, :, None]), dim=2)
    u = (window.float() * s["conv_weight"]).sum(2) + s["conv_bias"]
    u = u / (1.0 + torch.exp(-u))
    raw = s["dt"].float() + s["dt_bias"]
    dt = torch.clamp(raw, min=0.0) + torch.log1p(torch.exp(-raw.abs()))
    x = u[:, :d].view(batch, groups, -1, 64, 1)
    b = u[:, d:d + groups * n].view(batch, groups, 1, 1, n)
    c = u[:, d + groups * n:].view(batch, groups, 1, 1, n)
    step = dt.view(batch, groups, -1, 1, 1)
    h = s["state"][at].view(batch, groups, -1, 64, n)
    h = h * torch.exp(step * s["A"].view(groups, -1, 1, 1)) + step * x * b
    y = (h * c).sum(4) + s["D"].view(groups, -1, 1) * x[..., 0]
    z = s["z"].float()
    out = (y.reshape(batch, d) * (z / (1.0 + torch.exp(-z)))).to(s["xbc"].dtype)
    s["state"][at] = h.reshape(batch, d, n)
    s["conv_state"][at] = window[:, :, 1:]
    return out, s["state"], s["conv_state"]


_PLAIN = {
    "norm": _plain_norm,
    "norm_bwd": _plain_norm_bwd,
    "matmul": lambda s: _matmul(s["a"], s["a_scales"], s["b"], s["b_scales"],
                                DTYPES[s["case"]["out"]]),
    "linear": lambda s: _matmul(*_quantize(s["x"]), s["b"], s["b_scales"], DTYPES[s["case"]["out"]]),
    "linear_bwd": _plain_linear_bwd,
    "sample": _plain_sample,
    "step": _plain_step,
}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import selective_state_space_52_amd as mssm
    case = s["case"]
    op = case["op"]
    if op == "norm" and case["quantize"]:
        q, scales, stream, _ = mssm.rms_norm_fwd_fp8(s["x"], s["weight"], residual=s["residual"],
                                                     eps=s["eps"])
        return q, scales, stream
    if op == "norm":
        out, stream, _ = mssm.rms_norm_fwd(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
        return out, stream
    if op == "norm_bwd":
        return mssm.rms_norm_bwd(s["dout"], s["r"], s["weight"], s["rstd"], dresidual=s["dresidual"])
    if op == "matmul":
        return mssm.fp8_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"],
                               out_dtype=DTYPES[case["out"]])
    if op == "linear":
        q, scales = mssm.quantize_fp8(s["x"])
        return mssm.fp8_matmul(q, scales, s["b"], s["b_scales"], out_dtype=DTYPES[case["out"]])
    if op == "linear_bwd":
        g, g_scales = mssm.quantize_fp8(s["dout"])
        dx = mssm.fp8_matmul(g, g_scales, s["wt"], s["wt_scales"], out_dtype=s["x"].dtype)
        gt, gt_scales = mssm.quantize_fp8(s["dout"], transpose=True)
        xt, xt_scales = mssm.quantize_fp8(s["x"], transpose=True)
        return dx, mssm.fp8_matmul(gt, gt_scales, xt, xt_scales, out_dtype=torch.float32)
    if op == "sample":
        return mssm.sample_tokens(s["logits"], s["noise"], temperature=s["temperature"],
                                  top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    out = mssm.mamba2_state_update(s["state"], s["conv_state"], s["xbc"], s["dt"], s["conv_weight"],
                                   s["A"], conv_bias=s["conv_bias"], D=s["D"], z=s["z"],
                                   dt_bias=s["dt_bias"], ngroups=case["groups"], slots=s["slots"])
    return out, s["state"], s["conv_state"]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- floors

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op == "norm":
        io, res = size[case["io"]], size[case["res"]]
        out = 1 + 1 / BLOCK if case["quantize"] else io
        e = case["rows"] * case["dim"]
        return {"bytes": e * (io + 2 * res + out) + 4 * case["dim"], "flops": 6 * e}
    if op == "norm_bwd":
        io, res = size[case["io"]], size[case["res"]]
        e = case["rows"] * case["dim"]
        r = res if res else io
        return {"bytes": e * (2 * io + r + 2 * res) + 8 * case["dim"] + 4 * case["rows"],
                "flops": 10 * e}
    if op in ("matmul", "linear", "linear_bwd"):
        m, n, k = case["m"], case["n"], case["k"]
        weight = n * k + n * k / BLOCK ** 2
        if op == "linear_bwd":
            io = size[case["io"]]
            return {"bytes": io * (m * n + 2 * m * k) + weight + 4 * n * k, "flops": 4 * m * n * k}
        left = m * k * (1 + 1 / BLOCK) if op == "matmul" else m * k * size[case["io"]]
        return {"bytes": left + weight + m * n * size[case["out"]], "flops": 2 * m * n * k}
    if op == "sample":
        rows, vocab = case["rows"], case["vocab"]
        kept = min(vocab, case["top_k"]) if case["top_k"] else vocab
        return {"bytes": rows * (vocab * size[case["io"]] + 4 * kept + 12), "flops": 4 * rows * vocab}
    io, d, n = size[case["io"]], case["heads"] * 64, case["n"]
    ch = d + 2 * case["groups"] * n
    each = 8 * d * n + io * (7 * ch + 2 * d + case["heads"])
    return {"bytes": case["batch"] * each + 20 * ch + 12 * case["heads"],
            "flops": case["batch"] * (6 * d * n + 8 * ch)}


# ---------------------------------------------------------------- the same in 64 bits

def _exact_values(x, rows=1):
    """What e4m3 with power-of-two scales makes of x, and x / scale before its rounding."""
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // BLOCK)
    v = torch.zeros(mb * rows, kb * BLOCK, dtype=torch.float64, device=x.device)
    v[:m, :k] = x
    amax = v.abs().reshape(mb, rows, kb, BLOCK).permute(0, 2, 1, 3).reshape(mb, kb, -1).max(2).values
    scale = torch.exp2(torch.ceil(torch.log2(amax / FP8_MAX)).clamp(min=-127.0))
    wide = scale.repeat_interleave(rows, 0).repeat_interleave(BLOCK, 1)
    ratio = (v / wide)[:m, :k]
    return ratio.to(F8).double() * wide[:m, :k], ratio, scale


def _exact_scales(scales, rows, cols):
    v = scales.double()
    i = torch.arange(rows, device=v.device)
    j = torch.arange(cols, device=v.device) // BLOCK
    i = i if v.shape[0] == rows else i // BLOCK
    return v[i][:, j]


def _exact_norm(s):
    r = s["x"].double()
    stream = None
    if s["residual"] is not None:
        r = stream = r + s["residual"].double()
    y = s["weight"].double() * r / torch.sqrt((r ** 2).sum(1, keepdim=True) / r.shape[1] + s["eps"])
    if not s["case"]["quantize"]:
        return y, stream
    _, ratio, scale = _exact_values(y)
    return ratio, scale, stream


def _exact_norm_bwd(s):
    r, w, dy = s["r"].double(), s["weight"].double(), s["dout"].double()
    rstd = s["rstd"].double().unsqueeze(1)
    dot = (dy * w * r).sum(1, keepdim=True)
    dr = rstd * w * dy - rstd ** 3 * r * dot / r.shape[1]
    stream = None
    if s["dresidual"] is not None:
        dr = stream = dr + s["dresidual"].double()
    return dr, stream, (dy * r * rstd).sum(0)


def _exact_sample(s):
    tokens, logprobs = [], []
    for i in range(s["logits"].shape[0]):
        v = {name: float(s[name][i]) if isinstance(s[name], torch.Tensor) else float(s[name])
             for name in ("temperature", "top_k", "top_p", "min_p")}
        logit = s["logits"][i].double()
        if v["temperature"] == 0.0:
            tokens.append((logit == logit.max()).nonzero()[0, 0])
            logprobs.append(torch.zeros((), dtype=torch.float64, device=logit.device))
            continue
        order = torch.argsort(logit, descending=True, stable=True)
        order = order[:int(v["top_k"])] if v["top_k"] > 0 else order
        p = torch.softmax(logit[order] / v["temperature"], 0)
        if v["top_p"] < 1.0:
            ahead = torch.cat((p.new_zeros(1), torch.cumsum(p, 0)[:-1]))
            count = max(1, int((ahead < v["top_p"]).sum()))
            order, p = order[:count], p[:count]
        stay = p >= v["min_p"] * p[0]
        stay[0] = True
        order, p = order[stay], p[stay] / p[stay].sum()
        score = p / -torch.log(s["noise"][i].double()[order])
        top = order[score == score.max()].min()
        tokens.append(top)
        logprobs.append(torch.log(p[order == top][0]))
    return torch.stack(tokens), torch.stack(logprobs)


def _exact_step(s):
    case = s["case"]
    batch, heads, n, groups = case["batch"], case["heads"], case["n"], case["groups"]
    d = heads * 64
    rows = torch.arange(batch, device="cuda") if s["slots"] is None else s["slots"].long()
    past, new = s["conv_state"].double(), s["xbc"].double()
    cw = s["conv_weight"].double()
    u = s["conv_bias"].double() + cw[:, 3] * new
    for tap in range(3):
        u = u + cw[:, tap] * past[rows, :, tap]
    u = u * torch.sigmoid(u)
    dt = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=1e9)
    dt = dt.repeat_interleave(64, 1)                                   # per channel
    a = s["A"].double().repeat_interleave(64)
    group = torch.arange(d, device="cuda") // (d // groups)
    b = u[:, d:d + groups * n].reshape(batch, groups, n)
    c = u[:, d + groups * n:].reshape(batch, groups, n)
    state = s["state"].double()
    out = torch.empty(batch, d, dtype=torch.float64, device="cuda")
    for i in range(batch):
        h = torch.exp(dt[i] * a).unsqueeze(1) * state[rows[i]] + (dt[i] * u[i, :d]).unsqueeze(1) * b[i][group]
        y = (h * c[i][group]).sum(1) + s["D"].double().repeat_interleave(64) * u[i, :d]
        gate = s["z"][i].double()
        out[i] = y * gate * torch.sigmoid(gate)
        state[rows[i]] = h
    window = past.clone()
    window[rows, :, 0], window[rows, :, 1], window[rows, :, 2] = past[rows, :, 1], past[rows, :, 2], new
    return out, state, window


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_bwd":
        return _exact_norm_bwd(s)
    if op == "sample":
        return _exact_sample(s)
    if op == "step":
        return _exact_step(s)
    if op == "linear_bwd":
        dy, x = s["dout"].double(), s["x"].double()
        wt = s["wt"].double() * _exact_scales(s["wt_scales"], *s["wt"].shape)
        left = _exact_values(dy.t().contiguous())[0]
        right = _exact_values(x.t().contiguous())[0]
        return _exact_values(dy)[0] @ wt.t(), left @ right.t()
    if op == "linear":
        a = _exact_values(s["x"].double())[0]
    else:
        a = s["a"].double() * _exact_scales(s["a_scales"], *s["a"].shape)
    return a @ (s["b"].double() * _exact_scales(s["b_scales"], *s["b"].shape)).t()
