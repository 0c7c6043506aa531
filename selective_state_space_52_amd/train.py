"""The ends of a training step: the embedding's rows and their gradient, the
log-probabilities of given tokens with the policy and preference losses on them,
and the AdamW step.

A thin binding over the C ABI, like the layer's: tensors are checked, their
device pointers and the current HIP stream passed on.
"""
from __future__ import annotations

import struct

import torch

from ._lib import AdamwArgs, EmbedDims, LogprobDims, PolicyArgs, PreferenceArgs, lib
from .layer import _IO, F8, _call, _empty, _io, _is, _ptr, _rows, _size

__all__ = ["embedding_fwd", "embedding_bwd", "token_logprobs_fwd", "token_logprobs_bwd",
           "policy_loss", "preference_loss", "adamw_state", "adamw_step"]


def _dtype(dtype, name):
    if dtype not in _IO:
        raise ValueError("%s must be float32 or bfloat16" % name)
    return _IO[dtype]


def _empty1(n, device):
    return torch.empty_strided((n,), (1,), dtype=torch.float32, device=device)


def _tokens(tokens, device=None):
    if tokens.dim() != 1:
        raise ValueError("tokens must have 1 dimension")
    _is(tokens, "tokens", torch.int64, tokens.shape, tokens.device if device is None else device)
    if not tokens.is_cuda:
        raise ValueError("tokens must be a GPU tensor")
    return tokens.shape[0]


def embedding_fwd(tokens, table, scale=1.0, out_dtype=None):
    """Rows of an embedding table: scale * table[tokens].

    tokens: (rows,) int64; table: (vocab, dim) fp32 or bf16.  A token outside the
    table (the -1 of sample_tokens, say) is padding: its row is zero.  Returns
    (rows, dim) in out_dtype (fp32 or bf16; the table's by default)."""
    t = _io(table, "table", 2)
    dev = table.device
    rows = _tokens(tokens, dev)
    _is(table, "table", table.dtype, table.shape, dev)
    vocab, dim = table.shape
    out_dtype = table.dtype if out_dtype is None else out_dtype
    dims = EmbedDims(rows, vocab, dim, 0, t, _dtype(out_dtype, "out_dtype"), scale, 0)
    out = _empty(rows, dim, out_dtype, dev)
    _call(dev, lib().mssm_embedding_fwd, _ptr(tokens), _ptr(table), _ptr(out), dims)
    return out


# The most rows whose gradient needs no workspace.
_UNSORTED = 512


def embedding_bwd(tokens, dout, vocab, scale=1.0, out_dtype=torch.float32, add_to=None):
    """The table's gradient for dout (rows, dim) = dLoss/d(embedding_fwd), fp32 or
    bf16 with contiguous rows: scale times the sum of each token's rows.

    Returns (vocab, dim) in out_dtype (fp32 or bf16).  add_to: a gradient of that
    shape, fp32 or bf16, to which the sums are added in place (the one of an
    output projection that shares the table); it is returned.  Rows of padding
    give nothing.  Sums are fp32 in a fixed order."""
    io = _io(dout, "dout", 2)
    rows, dim = dout.shape
    dev = dout.device
    if _tokens(tokens, dev) != rows:
        raise ValueError("tokens has %d rows, dout %d" % (tokens.shape[0], rows))
    stride = _rows(dout, "dout", dout.dtype, dout.shape, dev)
    if add_to is None:
        t = _dtype(out_dtype, "out_dtype")
    else:
        t = _io(add_to, "add_to", 2)
        _is(add_to, "add_to", add_to.dtype, (vocab, dim), dev)
    dims = EmbedDims(rows, vocab, dim, stride, t, io, scale, int(add_to is not None))
    need = 0 if rows <= _UNSORTED else _size(lib().mssm_embedding_bwd_workspace, dims, dev)
    out = _empty(vocab, dim, out_dtype, dev) if add_to is None else add_to
    # from torch's caching allocator: ordered on the current stream, 512-byte aligned
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call(dev, lib().mssm_embedding_bwd, _ptr(tokens), _ptr(dout), _ptr(out), _ptr(ws), need, dims)
    return out


def _vector(t, name, rows, device):
    _is(t, name, torch.float32, (rows,), device)


def _logits(logits, tokens, temperature, out=None):
    """(dims, dlogits) of a call on these logits; dlogits is `out` if given."""
    io = _io(logits, "logits", 2)
    rows, vocab = logits.shape
    dev = logits.device
    stride = _rows(logits, "logits", logits.dtype, logits.shape, dev)
    if _tokens(tokens, dev) != rows:
        raise ValueError("tokens has %d rows, logits %d" % (tokens.shape[0], rows))
    grad_stride = 0 if out is None else _rows(out, "out", logits.dtype, logits.shape, dev)
    return LogprobDims(rows, vocab, stride, grad_stride, io, temperature)


# The longest rows whose sums need no workspace.
_WHOLE = 65536


def _parts(dims, device):
    """(workspace, bytes) of a call that sums rows of this length."""
    if dims.vocab <= _WHOLE:
        return None, 0
    need = _size(lib().mssm_token_logprobs_workspace, dims, device)
    return torch.empty(need, dtype=torch.uint8, device=device), need


def token_logprobs_fwd(logits, tokens, temperature=1.0):
    """Log-probabilities of tokens (rows,) int64 under softmax(logits /
    temperature); logits: (rows, vocab) fp32 or bf16 with contiguous rows.

    A token outside the vocabulary marks a row without one (a prompt's): its
    log-probability is 0.  Returns (logprobs (rows,) fp32, stats (rows, 2) fp32,
    which token_logprobs_bwd needs)."""
    dims = _logits(logits, tokens, temperature)
    dev, rows = logits.device, logits.shape[0]
    logprobs = _empty1(rows, dev)
    stats = _empty(rows, 2, torch.float32, dev)
    ws, need = _parts(dims, dev)
    _call(dev, lib().mssm_token_logprobs_fwd, _ptr(logits), _ptr(tokens), _ptr(logprobs),
          _ptr(stats), _ptr(ws), need, dims)
    return logprobs, stats


def token_logprobs_bwd(logits, tokens, stats, dlogprobs, temperature=1.0, out=None):
    """Gradient of token_logprobs_fwd's logprobs by the logits for dlogprobs
    (rows,) fp32.  Returns (rows, vocab) in the logits' dtype, or out (which may
    be logits itself, replaced by its gradient)."""
    dims = _logits(logits, tokens, temperature, out)
    dev, (rows, vocab) = logits.device, logits.shape
    _is(stats, "stats", torch.float32, (rows, 2), dev)
    _vector(dlogprobs, "dlogprobs", rows, dev)
    if out is None:
        out = _empty(rows, vocab, logits.dtype, dev)
    _call(dev, lib().mssm_token_logprobs_bwd, _ptr(logits), _ptr(tokens), _ptr(stats),
          _ptr(dlogprobs), _ptr(out), dims)
    return out


def policy_loss(logits, tokens, old_logprobs, advantages, ref_logprobs=None, weights=None,
                temperature=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.0, want_grad=True,
                out=None):
    """Clipped policy loss with a KL term, and its gradient by the logits.

    With logp the tokens' log-probabilities (token_logprobs_fwd) and ratio =
    exp(logp - old_logprobs), per row: -min(ratio A, clip(ratio, 1 - clip_low,
    1 + clip_high) A) + kl_coef (exp(x) - 1 - x), x = ref_logprobs - logp, A the
    advantage.  old_logprobs, advantages, ref_logprobs (None: no KL term) and
    weights (None: 1) are (rows,) fp32.  Rows whose token lies outside the
    vocabulary (a prompt's) have loss and logp 0 and a zero gradient.

    Returns (loss (rows,) fp32, logprobs (rows,) fp32, dlogits): dlogits is the
    gradient of sum(weights * loss) in the logits' dtype, written to out where
    given (which may be logits itself), None without want_grad."""
    if not want_grad and out is not None:
        raise ValueError("out is for the gradient, which is not wanted")
    dims = _logits(logits, tokens, temperature, out)
    dev, (rows, vocab) = logits.device, logits.shape
    _vector(old_logprobs, "old_logprobs", rows, dev)
    _vector(advantages, "advantages", rows, dev)
    if ref_logprobs is not None:
        _vector(ref_logprobs, "ref_logprobs", rows, dev)
    if weights is not None:
        _vector(weights, "weights", rows, dev)
    if want_grad and out is None:
        out = _empty(rows, vocab, logits.dtype, dev)
    loss, logprobs = _empty1(rows, dev), _empty1(rows, dev)
    ws, need = _parts(dims, dev)
    args = PolicyArgs(dims, clip_low, clip_high, kl_coef, 0)
    _call(dev, lib().mssm_policy_loss, _ptr(logits), _ptr(tokens), _ptr(old_logprobs),
          _ptr(advantages), _ptr(ref_logprobs), _ptr(weights), _ptr(loss), _ptr(logprobs),
          _ptr(out), _ptr(ws), need, args)
    return loss, logprobs, out


def preference_loss(logprobs, ref_logprobs, offsets, weights=None, beta=0.1, label_smoothing=0.0):
    """Preference loss of pairs of packed sequences, and its gradient.

    logprobs, ref_logprobs: (rows,) fp32, the tokens' log-probabilities under the
    policy and the reference (0 in a prompt's rows); offsets: (2 pairs + 1,)
    int32, sequence s having rows offsets[s] to offsets[s + 1] - 1, pair p being
    sequences 2p (preferred) and 2p + 1.  With d = beta times the difference of
    the two sums of logprobs - ref_logprobs: -(1 - label_smoothing) log sigmoid(d)
    - label_smoothing log sigmoid(-d).  weights: (pairs,) fp32, or None (1).
    Returns (loss (pairs,) fp32, dlogprobs (rows,) fp32, the gradient of
    sum(weights * loss), for token_logprobs_bwd)."""
    if logprobs.dim() != 1 or offsets.dim() != 1 or offsets.shape[0] < 3 or offsets.shape[0] % 2 == 0:
        raise ValueError("logprobs must be (rows,) and offsets (2 pairs + 1,)")
    dev, rows, pairs = logprobs.device, logprobs.shape[0], offsets.shape[0] // 2
    if not logprobs.is_cuda:
        raise ValueError("logprobs must be a GPU tensor")
    _vector(logprobs, "logprobs", rows, dev)
    _vector(ref_logprobs, "ref_logprobs", rows, dev)
    _is(offsets, "offsets", torch.int32, offsets.shape, dev)
    if weights is not None:
        _vector(weights, "weights", pairs, dev)
    loss, dlogprobs = _empty1(pairs, dev), _empty1(rows, dev)
    args = PreferenceArgs(rows, pairs, beta, label_smoothing)
    _call(dev, lib().mssm_preference_loss, _ptr(logprobs), _ptr(ref_logprobs), _ptr(offsets),
          _ptr(weights), _ptr(loss), _ptr(dlogprobs), args)
    return loss, dlogprobs


def adamw_state(params, bits=32):
    """Zero states for adamw_step of these tensors (none of them empty): (m, v,
    m_scales, v_scales).

    Each tensor's states begin at a multiple of 128 elements behind the last
    one's.  bits 32: m and v fp32, no scales (None); 8: float8_e4m3fn values and
    an fp32 scale for each 128 of them, m = value * scale and sqrt(v) = value *
    scale."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    if not params:
        raise ValueError("params is empty")
    if not all(p.numel() for p in params):
        raise ValueError("a tensor of params is empty: adamw_step takes none")
    dev = params[0].device
    n = sum(-(-p.numel() // 128) for p in params)
    if bits == 32:
        return (torch.zeros(n * 128, device=dev), torch.zeros(n * 128, device=dev), None, None)
    # zeros of an 8-bit float type: the bytes
    m, v = (torch.zeros(n * 128, dtype=torch.uint8, device=dev).view(F8) for _ in range(2))
    return m, v, torch.zeros(n, device=dev), torch.zeros(n, device=dev)


def _one(v, name, dtype, device):
    """A one-element tensor's pointer."""
    if v.numel() != 1:
        raise ValueError("%s must have one element" % name)
    _is(v, name, dtype, v.shape, device)
    return v.data_ptr()


def _plain(tensors, device):
    """Whether all are contiguous and on this device."""
    n = len(tensors)
    return (list(map(torch.Tensor.get_device, tensors)).count(device.index) == n
            and list(map(torch.Tensor.is_contiguous, tensors)).count(True) == n)


def _refuse_tensors(params, grads, device):
    for i, (p, g) in enumerate(zip(params, grads)):
        _is(p, "params[%d]" % i, torch.float32, p.shape, device)
        _io(g, "grads[%d]" % i, p.dim())
        _is(g, "grads[%d]" % i, g.dtype, p.shape, device)
    raise ValueError("params and grads do not fit together")


def _copies(copies, params, device):
    for i, (c, p) in enumerate(zip(copies, params)):
        if c is not None:
            _is(c, "copies[%d]" % i, torch.bfloat16, p.shape, device)
    return [0 if c is None else c.data_ptr() for c in copies]


def adamw_step(params, grads, m, v, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
               m_scales=None, v_scales=None, copies=None, grad_scale=1.0, seed=0):
    """AdamW step of many tensors, in place, in one launch for each 64 of them.

    params: fp32 tensors; grads: fp32 or bf16, of the same shapes; all
    contiguous, none empty.  m, v, m_scales, v_scales: as adamw_state gives them, for these
    tensors in this order.  step: 1, 2, ...; weight_decay: a number or one for
    each tensor; copies: None, or bf16 tensors (or None) that receive the new
    params; grad_scale multiplies the gradients (1 / loss scale, a clipping
    factor); seed: of the 8-bit states' rounding, which also goes by the step.
    lr, grad_scale (fp32) and step (int64) may be one-element GPU tensors, which a
    captured graph reads in every replay."""
    count = len(params)
    if count == 0 or len(grads) != count or (copies is not None and len(copies) != count):
        raise ValueError("params, grads and copies must be lists of the same length, not empty")
    f32 = torch.float32
    dev = params[0].device
    if not params[0].is_cuda:
        raise ValueError("params[0] must be a GPU tensor")
    decays = weight_decay if isinstance(weight_decay, (list, tuple)) else [weight_decay] * count
    if len(decays) != count:
        raise ValueError("weight_decay must be a number or one for each tensor")
    # lists and maps: half the time of a loop over the tensors
    codes = list(map(_IO.get, [g.dtype for g in grads]))
    if not (_plain(params, dev) and _plain(grads, dev) and None not in codes
            and [p.dtype for p in params].count(f32) == count
            and [p.shape for p in params] == [g.shape for g in grads]):
        _refuse_tensors(params, grads, dev)
    sizes = list(map(torch.Tensor.numel, params))
    blocks = sum([(n + 127) >> 7 for n in sizes])
    flat = [None] * (6 * count)     # mssm_adamw_tensor's fields
    flat[0::6] = map(torch.Tensor.data_ptr, params)
    flat[1::6] = map(torch.Tensor.data_ptr, grads)
    flat[2::6] = [0] * count if copies is None else _copies(copies, params, dev)
    flat[3::6], flat[4::6], flat[5::6] = sizes, decays, codes
    table = struct.pack("PPPqfi" * count, *flat)
    eight = m.dtype is F8
    for t, name in ((m, "m"), (v, "v")):
        _is(t, name, F8 if eight else f32, (blocks * 128,), dev)
    for t, name in ((m_scales, "m_scales"), (v_scales, "v_scales")):
        if eight != (t is not None):
            raise ValueError("%s belongs to states in 8 bits, and only to those" % name)
        if eight:
            _is(t, name, f32, (blocks,), dev)
    args = AdamwArgs(beta1=betas[0], beta2=betas[1], eps=eps, seed=seed & (2 ** 64 - 1),
                     state_bits=8 if eight else 32)
    if isinstance(lr, torch.Tensor):
        args.lr_value = _one(lr, "lr", f32, dev)
    else:
        args.lr = lr
    if isinstance(grad_scale, torch.Tensor):
        args.grad_scale_value = _one(grad_scale, "grad_scale", f32, dev)
    else:
        args.grad_scale = grad_scale
    if isinstance(step, torch.Tensor):
        args.step_value = _one(step, "step", torch.int64, dev)
    else:
        args.step = step
    _call(dev, lib().mssm_adamw, table, count, _ptr(m), _ptr(v), _ptr(m_scales), _ptr(v_scales), args)
