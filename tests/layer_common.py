"""64-bit references of the layer's operators around the scans, on the CPU or
the GPU, and the tolerances of their tests.

Tolerances.  U32 = 2^-24 and U16 = 2^-8 (24 and 8 significant bits) are the relative roundings of fp32 and
bf16.  A sum of n terms in fp32 is within (n + 4) U32 sum|term| of its value in
any order; a hardware exp2, log2, rsqrt or reciprocal within 4 U32.  A result
that is rounded to bf16 adds U16 |result|.
"""
import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {torch.bfloat16: U16, torch.float32: U32}


def bound(got, ref, slack, dtype):
    """|got - ref| <= slack + one rounding to the result's type, where finite."""
    got, ref = got.double().cpu(), ref.double().cpu()
    slack = slack.double().cpu() if isinstance(slack, torch.Tensor) else slack
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    limit = slack + 1.01 * ROUND[dtype] * (ref.abs() + slack)
    err = (got - ref).abs()
    fine = torch.isnan(ref) | (got == ref) | (err <= limit)
    assert fine.all(), "worst excess %.3g at %s" % (
        float((err - limit)[~fine].max()), (~fine).nonzero()[0].tolist())


def exp2i(code):
    return torch.exp2(code.double() - 127.0)


def quantize(x, block_rows=1):
    """e4m3 values, e8m0 codes and what they stand for, in 64 bits, block by
    block (no torch rounding but the one to e4m3)."""
    rows, cols = x.shape
    q = torch.zeros(rows, cols, dtype=F8)
    codes = torch.zeros(-(-rows // block_rows), -(-cols // 128), dtype=torch.uint8)
    for i in range(codes.shape[0]):
        for j in range(codes.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            v = x[at].double()
            fine = torch.isfinite(v)
            amax = float(v[fine].abs().max()) if fine.any() else 0.0
            code = 0
            while code < 254 and amax > 448.0 * 2.0 ** (code - 127):
                code += 1
            codes[i, j] = code
            q[at] = torch.where(fine, v * 2.0 ** (127 - code), torch.nan).float().to(F8)
    return q, codes


def widen(q, codes, block_rows=1):
    rows, cols = q.shape
    s = exp2i(codes).repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q.double() * s


def rms_norm(x, weight, residual, eps):
    r = x.double() if residual is None else x.double() + residual.double()
    rstd = 1.0 / torch.sqrt((r * r).mean(1) + eps)
    return r * rstd[:, None] * weight.double(), r, rstd


def rms_norm_bwd(dout, r, weight, rstd, dresidual):
    g, r, w, s = dout.double(), r.double(), weight.double(), rstd.double()[:, None]
    xhat = r * s
    dr = s * (w * g - xhat * (w * g * xhat).mean(1, keepdim=True))
    return (dr if dresidual is None else dr + dresidual.double()), (g * xhat).sum(0)


def sample(logits, noise, temperature, top_k, top_p, min_p):
    """One row at a time, as the definition reads."""
    tokens, logprobs = [], []
    for i in range(logits.shape[0]):
        l, u = logits[i].double(), noise[i].double()
        l = torch.where(torch.isnan(l), -torch.inf, l)
        m = l.max()
        if m == -torch.inf:
            tokens.append(-1)
            logprobs.append(float("-inf"))
            continue
        order = torch.argsort(l, descending=True, stable=True)
        if not temperature[i] > 0:
            tokens.append(int(order[0]))
            logprobs.append(0.0)
            continue
        w = torch.where(l == m, 1.0, torch.exp((l - m) / temperature[i]))
        if top_k[i] > 0:
            order = order[:int(top_k[i])]
        if top_p[i] < 1:
            mass = w[order]
            before = torch.cumsum(mass, 0) - mass
            stay = before < top_p[i] * mass.sum()
            stay[0] = True
            order = order[stay]
        stay = (w[order] >= min_p[i]) & (w[order] > 0)
        stay[0] = True
        order = order[stay].sort().values
        e = torch.where(u[order] > 0, -torch.log(u[order]), torch.inf)
        score = torch.where(e > 0, w[order] / e, torch.inf)
        token = int(order[(score == score.max()).nonzero()[0, 0]])
        tokens.append(token)
        scaled = 0.0 if l[token] == m else float((l[token] - m) / temperature[i])
        logprobs.append(scaled - float(torch.log(w[order].sum())))
    return tokens, logprobs


def mamba2_step(state, conv_state, xbc, dt, conv_weight, A, conv_bias, D, z, dt_bias, softplus,
                ngroups, slots, sizes=False):
    """Returns out, state, conv_state in 64 bits, sequence by sequence; with
    `sizes`, the sums of the absolute values of the terms of each instead (the
    decay as it is): what a rounding of each term is relative to."""
    state, conv_state = state.double().clone(), conv_state.double().clone()
    if sizes:
        state = state.abs()
    batch, heads = dt.shape
    N, dim = state.shape[2], heads * 64
    out = torch.zeros(batch, dim, dtype=torch.float64)
    for b in range(batch):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < state.shape[0]:
            continue
        v = torch.cat((conv_state[s], xbc[b].double()[:, None]), 1)
        u = v * conv_weight.double()
        u = torch.cat((u, torch.zeros(u.shape[0], 1) if conv_bias is None
                       else conv_bias.double()[:, None]), 1)
        u = u.abs().sum(1) if sizes else u.sum(1) * torch.sigmoid(u.sum(1))
        conv_state[s] = v[:, 1:]
        B = u[dim:dim + ngroups * N].view(ngroups, N)
        C = u[dim + ngroups * N:].view(ngroups, N)
        for h in range(heads):
            g, at = h // (heads // ngroups), slice(h * 64, h * 64 + 64)
            step = dt[b, h].double() + (0.0 if dt_bias is None else dt_bias[h].double())
            if softplus:
                step = torch.log1p(torch.exp(-step.abs())) + step.clamp(min=0)
            x = u[at]
            state[s, at] = torch.exp(step * A[h].double()) * state[s, at] + step * x[:, None] * B[g]
            skip = 0.0 if D is None else D[h].double()
            y = state[s, at] @ C[g] + (abs(skip) if sizes else skip) * x
            if z is not None:
                gate = z[b, at].double() * torch.sigmoid(z[b, at].double())
                y = y * (gate.abs() if sizes else gate)
            out[b, at] = y
    return out, state, conv_state
