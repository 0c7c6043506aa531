"""The layer around the scans: the norm that joins the residual stream (its
output also in 8 bits), the 8-bit products and their quantiser, the Mamba-2
single-token step with its convolution, and the choice of the next token.

A thin binding over the C ABI, like the scans': tensors are checked, their
device pointers and the current HIP stream passed on.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import (MSSM_BF16, MSSM_F32, MatmulDims, NormDims, QuantDims, SampleArgs, StepDims,
                   check, lib)

__all__ = ["rms_norm_fwd", "rms_norm_fwd_fp8", "rms_norm_bwd", "quantize_fp8", "fp8_matmul",
           "sample_tokens", "mamba2_state_update"]

_IO = {torch.float32: MSSM_F32, torch.bfloat16: MSSM_BF16}
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _ptr(t):
    return None if t is None else t.data_ptr()


def _is(t, name, dtype, shape, device):
    """A contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dtype, shape, device)
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name, dtype, shape, device):
    """A tensor of rows, each contiguous; the elements from one to the next."""
    if t.dtype is not dtype or t.device != device or t.shape != shape:
        _refuse(t, name, dtype, shape, device)
    rows, cols = shape
    s = t.stride()
    if (cols > 1 and s[1] != 1) or (rows > 1 and s[0] < cols):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return s[0] if rows > 1 else cols


def _refuse(t, name, dtype, shape, device):
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _io(t, name, dims):
    io = _IO.get(t.dtype)
    if io is None:
        raise ValueError("%s must be float32 or bfloat16" % name)
    if t.dim() != dims:
        raise ValueError("%s must have %d dimensions" % (name, dims))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    return io


# The current device and its current stream's handle, without the Stream object
# that torch.cuda.current_stream makes (2 us of a small call's 14).
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(device, fn, *args):
    """fn(*args, current stream of the device), checked."""
    index = device.index
    if index == _current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(index))
    if rc:
        check(rc)


def _size(fn, dims, device):
    """Bytes of workspace that a call on this device needs."""
    n = ctypes.c_int64(0)
    if device.index == _current_device():
        check(fn(dims, n))
    else:
        with torch.cuda.device(device):
            check(fn(dims, n))
    return n.value


# The step's counters, one buffer for each (device, stream), on which calls run
# in order: cleared when it is made, left at zero by every call.
_COUNTERS = {}


def _counters(device, need):
    if torch.cuda.is_current_stream_capturing():
        # a graph's own, cleared in the graph: it may be replayed on any stream
        return torch.zeros(need // 4, dtype=torch.int32, device=device)
    key = (device.index, _raw_stream(device.index))
    buf = _COUNTERS.get(key)
    if buf is None or buf.numel() * 4 < need:
        buf = _COUNTERS[key] = torch.zeros(max(1024, need // 4), dtype=torch.int32, device=device)
    return buf


def _empty(rows, cols, dtype, device):
    # a fifth faster than torch.empty
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _norm(x, weight, residual, eps, want_rstd, fp8):
    io = _io(x, "x", 2)
    rows, dim = x.shape
    dev = x.device
    stride = _rows(x, "x", x.dtype, x.shape, dev)
    _is(weight, "weight", torch.float32, (dim,), dev)
    stream, res = None, io
    if residual is not None:
        res = _io(residual, "residual", 2)
        _is(residual, "residual", residual.dtype, x.shape, dev)
        stream = torch.empty_like(residual)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if want_rstd else None
    dims = NormDims(rows, dim, stride, io, res, eps, 0)
    if fp8:
        q = _empty(rows, dim, F8, dev)
        scales = _empty(rows, (dim + 127) // 128, E8, dev)
        _call(dev, lib().mssm_rms_norm_fwd_fp8, _ptr(x), _ptr(residual), _ptr(weight), _ptr(q),
              _ptr(scales), _ptr(stream), _ptr(rstd), dims)
        return q, scales, stream, rstd
    out = _empty(rows, dim, x.dtype, dev)
    _call(dev, lib().mssm_rms_norm_fwd, _ptr(x), _ptr(residual), _ptr(weight), _ptr(out),
          _ptr(stream), _ptr(rstd), dims)
    return out, stream, rstd


def rms_norm_fwd(x, weight, residual=None, eps=1e-5, want_rstd=False):
    """RMS norm of r = x + residual: r * weight / sqrt(mean(r^2) + eps).

    x: (rows, dim) fp32 or bf16, its rows contiguous; weight: (dim,) fp32;
    residual: (rows, dim) fp32 or bf16, or None (r = x).  Returns
    (out in x's dtype, r in the residual's dtype or None, rstd (rows,) fp32 or
    None): r is the residual stream of the next layer, and r and rstd are what
    rms_norm_bwd needs.
    """
    return _norm(x, weight, residual, eps, want_rstd, False)


def rms_norm_fwd_fp8(x, weight, residual=None, eps=1e-5, want_rstd=False):
    """rms_norm_fwd with its output in 8 bits, for fp8_matmul.  Returns (q
    (rows, dim) float8_e4m3fn, scales (rows, ceil(dim / 128)) float8_e8m0fnu,
    r or None, rstd or None)."""
    return _norm(x, weight, residual, eps, want_rstd, True)


def rms_norm_bwd(dout, r, weight, rstd, dresidual=None):
    """Gradients of rms_norm_fwd for dout (rows, dim) = dLoss/dout.

    r, rstd: what the forward call returned (r is x itself where it had no
    residual).  dresidual: the gradient of r from its later uses, in r's dtype,
    where there was a residual (zeros if it has none); None where there was
    not.  Returns (dx in dout's dtype, the residual's gradient in r's dtype or
    None without dresidual, dweight (dim,) fp32)."""
    io = _io(dout, "dout", 2)
    rows, dim = dout.shape
    dev = dout.device
    has = dresidual is not None
    _is(dout, "dout", dout.dtype, dout.shape, dev)
    res = _io(r, "r", 2) if has else io
    _is(r, "r", r.dtype if has else dout.dtype, dout.shape, dev)
    _is(weight, "weight", torch.float32, (dim,), dev)
    _is(rstd, "rstd", torch.float32, (rows,), dev)
    dr = None
    if has:
        _is(dresidual, "dresidual", r.dtype, dout.shape, dev)
        dr = torch.empty_like(r)
    dx = torch.empty_like(dout)
    dw = torch.empty(dim, dtype=torch.float32, device=dev)
    dims = NormDims(rows, dim, 0, io, res, 0.0, 0)
    need = _size(lib().mssm_rms_norm_bwd_workspace, dims, dev)
    # from torch's caching allocator: ordered on the current stream, 512-byte aligned
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(dev, lib().mssm_rms_norm_bwd, _ptr(dout), _ptr(r), _ptr(weight), _ptr(rstd),
          _ptr(dresidual), _ptr(dx), _ptr(dr), _ptr(dw), _ptr(ws), need, dims, int(has))
    return dx, dr, dw


def quantize_fp8(x, block_rows=1, transpose=False):
    """x (rows, cols), fp32 or bf16 with contiguous rows, in 8 bits.

    block_rows 1: a power-of-two scale for each 128 along a row of the result
    (activations, gradients); 128: one for each 128 x 128 block (weights).
    transpose: the result is x transposed.  Returns (q float8_e4m3fn, scales
    float8_e8m0fnu of shape (ceil(q rows / block_rows), ceil(q columns / 128))).
    """
    io = _io(x, "x", 2)
    rows, cols = x.shape
    stride = _rows(x, "x", x.dtype, x.shape, x.device)
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    qr, qc = (cols, rows) if transpose else (rows, cols)
    q = _empty(qr, qc, F8, x.device)
    scales = _empty(-(-qr // block_rows), -(-qc // 128), E8, x.device)
    dims = QuantDims(rows, cols, stride, io, block_rows, int(bool(transpose)), 0)
    _call(x.device, lib().mssm_quantize_fp8, _ptr(x), _ptr(q), _ptr(scales), dims)
    return q, scales


def fp8_matmul(a, a_scales, b, b_scales, out_dtype=torch.bfloat16, out=None):
    """a @ b.T of 8-bit values with a scale for each block of 128 along k.

    a: (M, K), b: (N, K) float8_e4m3fn; a_scales: (M, ceil(K / 128)), b_scales:
    (ceil(N / 128), ceil(K / 128)) or (N, ceil(K / 128)), float8_e8m0fnu, as
    quantize_fp8 and rms_norm_fwd_fp8 return them.  Returns (M, N) in out_dtype
    (bf16 or fp32), or out.  Sums are fp32; the products are exact for an fp32
    result, and for a bf16 one cut at 2^-13 of the largest of each 8 along k (see
    mssm_fp8_matmul in include/mssm.h).
    """
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must have 2 dimensions")
    (M, K), N, dev = a.shape, b.shape[0], a.device
    if not a.is_cuda:
        raise ValueError("a must be a GPU tensor")
    kb = -(-K // 128)
    _is(a, "a", F8, (M, K), dev)
    _is(b, "b", F8, (N, K), dev)
    _is(a_scales, "a_scales", E8, (M, kb), dev)
    rows = 1 if b_scales.dim() == 2 and b_scales.shape[0] == N and N > 1 else 128
    _is(b_scales, "b_scales", E8, (N if rows == 1 else -(-N // 128), kb), dev)
    if out is None:
        if out_dtype not in _IO:
            raise ValueError("out_dtype must be float32 or bfloat16")
        out = _empty(M, N, out_dtype, dev)
    else:
        _io(out, "out", 2)
        _is(out, "out", out.dtype, (M, N), dev)
    dims = MatmulDims(M, N, K, _IO[out.dtype], rows)
    _call(dev, lib().mssm_fp8_matmul, _ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales), _ptr(out),
          dims)
    return out


def sample_tokens(logits, noise, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The next token of each row of logits (rows, vocab), fp32 or bf16, from
    noise (rows, vocab) fp32 uniform on (0, 1); both with contiguous rows.

    temperature (0: the likeliest token), top_k (0: all), top_p and min_p are
    numbers, or (rows,) tensors (top_k int32, the others fp32).  Returns
    (tokens (rows,) int64, log-probabilities (rows,) fp32); see mssm_sample in
    include/mssm.h for the definition."""
    io = _io(logits, "logits", 2)
    rows, vocab = logits.shape
    dev = logits.device
    args = SampleArgs(rows, vocab, _rows(logits, "logits", logits.dtype, logits.shape, dev),
                      _rows(noise, "noise", torch.float32, logits.shape, dev), io)
    for name, v, dtype in (("temperature", temperature, torch.float32),
                           ("top_k", top_k, torch.int32),
                           ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(v, torch.Tensor):
            _is(v, name, dtype, (rows,), dev)
            setattr(args, name + "_row", v.data_ptr())
        elif name == "top_k":
            args.top_k = max(0, min(int(v), 2**31 - 1))     # ctypes would cut it to 32 bits
        else:
            setattr(args, name, v)
    tokens = torch.empty(rows, dtype=torch.int64, device=dev)
    logprobs = torch.empty(rows, dtype=torch.float32, device=dev)
    _call(dev, lib().mssm_sample, _ptr(logits), _ptr(noise), _ptr(tokens), _ptr(logprobs), args)
    return tokens, logprobs


def mamba2_state_update(state, conv_state, xbc, dt, conv_weight, A, conv_bias=None, D=None, z=None,
                        dt_bias=None, softplus=True, ngroups=1, slots=None, out=None):
    """Single-token step of a Mamba-2 block: the causal convolution (with silu)
    over the x, B and C channels, then the scan's step; state and conv_state are
    updated in place.

    state: (cache, nheads * 64, N) fp32 (the prompt's last_state), N 64 or 128;
    conv_state: (cache, channels, width - 1), channels = nheads * 64
    + 2 * ngroups * N; xbc: (batch, channels); dt: (batch, nheads); z: (batch,
    nheads * 64) or None; the last three may be columns of one projection's
    output.  conv_weight: (channels, width) fp32, conv_bias: (channels,) fp32 or
    None; A, D, dt_bias: (nheads,) fp32, D and dt_bias or None.  slots: (batch,)
    int32, each sequence's row of the states (no two alike; one outside the
    cache is padding: its out is zero), or None with cache = batch.  Returns out
    (batch, nheads * 64) in xbc's dtype (fp32 or bf16).
    """
    io = _io(xbc, "xbc", 2)
    dev, dtype = xbc.device, xbc.dtype
    batch, ch = xbc.shape
    if state.dim() != 3 or conv_weight.dim() != 2 or dt.dim() != 2:
        raise ValueError("state must be (cache, nheads * 64, N), conv_weight (channels, width), "
                         "dt (batch, nheads)")
    cache, dim, N = state.shape
    heads, width = dt.shape[1], conv_weight.shape[1]
    if dim != heads * 64 or ch != dim + 2 * ngroups * N:
        raise ValueError("state, dt, xbc and ngroups do not fit together: state %s, dt %s, xbc %s, "
                         "%d groups" % (tuple(state.shape), tuple(dt.shape), tuple(xbc.shape), ngroups))
    _is(state, "state", torch.float32, state.shape, dev)
    _is(conv_state, "conv_state", dtype, (cache, ch, width - 1), dev)
    _is(conv_weight, "conv_weight", torch.float32, (ch, width), dev)
    strides = [_rows(xbc, "xbc", dtype, xbc.shape, dev), _rows(dt, "dt", dtype, (batch, heads), dev),
               0 if z is None else _rows(z, "z", dtype, (batch, dim), dev)]
    _is(A, "A", torch.float32, (heads,), dev)
    for t, name, n in ((conv_bias, "conv_bias", ch), (D, "D", heads), (dt_bias, "dt_bias", heads)):
        if t is not None:
            _is(t, name, torch.float32, (n,), dev)
    if slots is not None:
        _is(slots, "slots", torch.int32, (batch,), dev)
    elif cache != batch:
        raise ValueError("state has %d rows for %d sequences: give slots" % (cache, batch))
    if out is None:
        out = _empty(batch, dim, dtype, dev)
    else:
        _is(out, "out", dtype, (batch, dim), dev)
    dims = StepDims(batch, cache, heads, 64, ngroups, N, *strides, width, io)
    need = batch * ngroups * 4
    ws = _counters(dev, need)
    _call(dev, lib().mssm_mamba2_state_update, _ptr(state), _ptr(conv_state), _ptr(xbc), _ptr(dt),
          _ptr(conv_weight), _ptr(conv_bias), _ptr(A), _ptr(D), _ptr(z), _ptr(dt_bias),
          int(bool(softplus)), _ptr(slots), _ptr(out), _ptr(ws), need, dims)
    return out
