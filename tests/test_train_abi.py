"""Refusals of the entry points of a training step's ends: every call below
fails validation, which happens before the first HIP call, so the pointers are
never read."""
import ctypes
import os

import pytest

from tests.test_layer_abi import ALIAS, ALIGN, BASE, BF16, DIMS, F32, NULL, UNSUPPORTED, far

WORKSPACE = -7


@pytest.fixture(scope="module")
def L():
    from selective_state_space_52_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from selective_state_space_52_amd import build
        build.build(force=True)
    return _lib.lib()


def _embed(rows=16, vocab=100, dim=64, stride=0, table=F32, io=BF16, scale=1.0, add=0):
    from selective_state_space_52_amd._lib import EmbedDims
    return EmbedDims(rows, vocab, dim, stride, table, io, scale, add)


BAD_EMBED = (dict(rows=0), dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 22) + 1),
             dict(dim=0), dict(dim=(1 << 20) + 1), dict(stride=63), dict(stride=1 << 62),
             dict(rows=1 << 30, dim=1 << 20))


def test_embedding_forward(L):
    names = ("tokens", "table", "out")
    p = far(names)

    def call(dims=None, **o):
        q = {**p, **o}
        return L.mssm_embedding_fwd(*[q[n] for n in names], dims or _embed(), None)
    assert L.mssm_embedding_fwd(*p.values(), None, None) == NULL
    for n in names:
        assert call(**{n: None}) == NULL, n
    for bad in BAD_EMBED:
        assert call(_embed(**bad)) == DIMS, bad
    for bad in (dict(table=2), dict(io=-1)):
        assert call(_embed(**bad)) == UNSUPPORTED, bad
    assert call(tokens=p["tokens"] + 4) == ALIGN
    assert call(table=p["table"] + 2) == ALIGN
    assert call(out=p["out"] + 1) == ALIGN
    assert call(out=p["table"] + 100 * 64 * 4 - 2) == ALIAS
    assert call(_embed(stride=80), out=p["tokens"] - 2 * (15 * 80 + 63)) == ALIAS


def test_embedding_backward(L):
    names = ("tokens", "dout", "dtable", "ws")
    p = far(names)

    def call(dims=None, size=1 << 30, **o):
        q = {**p, **o}
        return L.mssm_embedding_bwd(*[q[n] for n in names], size, dims or _embed(), None)
    n = ctypes.c_int64(0)
    assert L.mssm_embedding_bwd_workspace(_embed(rows=512), n) == 0 and n.value == 0
    many = dict(rows=513)
    assert L.mssm_embedding_bwd_workspace(_embed(**many), n) == 0 and n.value > 0
    need = n.value
    assert L.mssm_embedding_bwd_workspace(_embed(), None) == NULL
    assert L.mssm_embedding_bwd_workspace(None, n) == NULL
    for name in names[:3]:
        assert call(**{name: None}) == NULL, name
    for bad in BAD_EMBED:
        assert call(_embed(**bad)) == DIMS, bad
        assert L.mssm_embedding_bwd_workspace(_embed(**bad), n) == DIMS, bad
    assert call(_embed(io=3)) == UNSUPPORTED
    assert call(dout=p["dout"] + 1) == ALIGN
    assert call(dtable=p["dtable"] + 2) == ALIGN
    assert call(dtable=p["dout"] + 16 * 64 * 2 - 4) == ALIAS
    assert call(_embed(**many), ws=p["dtable"]) == ALIAS
    assert call(_embed(**many), ws=p["tokens"] - 256) == ALIAS
    assert call(_embed(**many), ws=None) == WORKSPACE
    assert call(_embed(**many), size=need - 1) == WORKSPACE
    assert call(_embed(**many), ws=p["ws"] + 16) == WORKSPACE


def _logp(rows=4, vocab=1000, ls=0, gs=0, io=BF16, t=1.0):
    from selective_state_space_52_amd._lib import LogprobDims
    return LogprobDims(rows, vocab, ls, gs, io, t)


BAD_LOGP = (dict(rows=0), dict(rows=1 << 22), dict(vocab=0), dict(vocab=(1 << 22) + 1), dict(ls=999),
            dict(ls=1 << 61), dict(t=0.0), dict(t=-1.0), dict(t=float("nan")), dict(t=float("inf")),
            dict(t=1e-40))


def test_token_logprobs(L):
    names = ("logits", "tokens", "logprobs", "stats")
    p = far(names)

    def call(dims=None, **o):
        q = {**p, **o}
        return L.mssm_token_logprobs_fwd(*[q[n] for n in names], ws, size, dims or _logp(), None)
    ws, size = None, 0
    assert L.mssm_token_logprobs_fwd(*p.values(), None, 0, None, None) == NULL
    for n in names[:3]:
        assert call(**{n: None}) == NULL, n
    for bad in BAD_LOGP:
        assert call(_logp(**bad)) == DIMS, bad
    assert call(_logp(io=4)) == UNSUPPORTED
    assert call(logits=p["logits"] + 1) == ALIGN
    assert call(tokens=p["tokens"] + 4) == ALIGN
    assert call(stats=p["stats"] + 2) == ALIGN
    assert call(stats=p["logprobs"] + 12) == ALIAS
    assert call(logprobs=p["logits"] + 4 * 1000 * 2 - 4) == ALIAS
    # the workspace of long rows
    n = ctypes.c_int64(-1)
    assert L.mssm_token_logprobs_workspace(_logp(vocab=65536), n) == 0 and n.value == 0
    assert L.mssm_token_logprobs_workspace(_logp(vocab=65537), n) == 0 and n.value == 4 * 19 * 4
    assert L.mssm_token_logprobs_workspace(_logp(rows=0), n) == DIMS
    assert L.mssm_token_logprobs_workspace(_logp(), None) == NULL
    long = _logp(vocab=65537)
    assert call(long) == WORKSPACE
    ws, size = BASE - 4096, 4 * 19 * 4 - 1
    assert call(long) == WORKSPACE
    ws, size = p["logprobs"], 1 << 20
    assert call(long) == ALIAS
    ws = BASE - 4096 + 4
    assert call(long) == WORKSPACE


def test_token_logprobs_backward(L):
    names = ("logits", "tokens", "stats", "dlogprobs", "dlogits")
    p = far(names)

    def call(dims=None, **o):
        q = {**p, **o}
        return L.mssm_token_logprobs_bwd(*[q[n] for n in names], dims or _logp(), None)
    for n in names:
        assert call(**{n: None}) == NULL, n
    for bad in BAD_LOGP + (dict(gs=10), dict(rows=(1 << 22) - 1, vocab=1 << 22)):
        assert call(_logp(**bad)) == DIMS, bad
    assert call(dlogits=p["dlogits"] + 1) == ALIGN
    assert call(dlogits=p["logits"] + 2) == ALIAS                 # in place only as a whole
    assert call(_logp(ls=1008, gs=1016), dlogits=p["logits"]) == ALIAS
    assert call(dlogits=p["stats"] + 28) == ALIAS


def _policy(low=0.2, high=0.2, kl=0.0, **o):
    from selective_state_space_52_amd._lib import PolicyArgs
    return PolicyArgs(_logp(**o), low, high, kl, 0)


def test_policy_loss(L):
    names = ("logits", "tokens", "old", "adv", "ref", "weights", "loss", "logprobs", "dlogits")
    p = far(names)

    def call(args=None, **o):
        q = {**p, **o}
        return L.mssm_policy_loss(*[q[n] for n in names], ws, size, args or _policy(), None)
    ws, size = None, 0
    assert L.mssm_policy_loss(*p.values(), None, 0, None, None) == NULL
    for n in ("logits", "tokens", "old", "adv", "loss", "logprobs"):
        assert call(**{n: None}) == NULL, n
    for bad in BAD_LOGP + (dict(gs=10), dict(low=-0.1), dict(high=float("nan")), dict(kl=-1.0),
                           dict(kl=float("inf"))):
        assert call(_policy(**bad)) == DIMS, bad
    assert call(old=p["old"] + 2) == ALIGN
    assert call(dlogits=p["logits"] + 64) == ALIAS
    assert call(loss=p["old"]) == ALIAS
    assert call(loss=p["logits"], dlogits=None) == ALIAS
    assert call(logprobs=p["dlogits"] + 8) == ALIAS
    assert call(_policy(vocab=70000)) == WORKSPACE
    ws, size = p["dlogits"] + 256, 1 << 20
    assert call(_policy(vocab=70000)) == ALIAS


def test_preference_loss(L):
    from selective_state_space_52_amd._lib import PreferenceArgs
    names = ("logprobs", "ref", "offsets", "weights", "loss", "dlogprobs")
    p = far(names)

    def call(args=None, **o):
        q = {**p, **o}
        return L.mssm_preference_loss(*[q[n] for n in names], args or PreferenceArgs(40, 3, 0.1, 0.0),
                                      None)
    assert L.mssm_preference_loss(*p.values(), None, None) == NULL
    for n in ("logprobs", "ref", "offsets", "loss", "dlogprobs"):
        assert call(**{n: None}) == NULL, n
    for bad in ((0, 3, 0.1, 0.0), (40, 0, 0.1, 0.0), (1 << 31, 3, 0.1, 0.0), (40, 1 << 21, 0.1, 0.0),
                (40, 3, float("nan"), 0.0), (40, 3, 0.1, -0.1), (40, 3, 0.1, 1.5)):
        assert call(PreferenceArgs(*bad)) == DIMS, bad
    assert call(offsets=p["offsets"] + 2) == ALIGN
    assert call(dlogprobs=p["logprobs"]) == ALIAS
    assert call(loss=p["offsets"] + 24) == ALIAS
    assert call(loss=p["dlogprobs"] + 156) == ALIAS


def test_adamw(L):
    from selective_state_space_52_amd._lib import AdamwArgs, AdamwTensor
    names = ("p0", "g0", "c0", "p1", "g1", "c1", "m", "v", "ms", "vs")
    p = far(names)

    def call(sizes=(300, 5), dtypes=(BF16, F32), bits=8, count=2, args=None, ptrs=None, **o):
        q = {**p, **(ptrs or {})}
        table = (AdamwTensor * 2)(*[(q["p%d" % i], q["g%d" % i], q["c%d" % i], sizes[i], 0.1, dtypes[i])
                                    for i in range(2)])
        a = AdamwArgs(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0, step=1,
                                state_bits=bits), **o})
        return L.mssm_adamw(table, count, q["m"], q["v"], q["ms"], q["vs"], a, None)
    none = dict(ms=None, vs=None)
    assert L.mssm_adamw(None, 1, p["m"], p["v"], None, None, AdamwArgs(state_bits=32), None) == NULL
    assert L.mssm_adamw((AdamwTensor * 1)(), 1, p["m"], p["v"], None, None, None, None) == NULL
    for n in ("p0", "g1", "m", "v", "ms", "vs"):
        assert call(ptrs={n: None}) == NULL, n
    assert call(bits=32) == UNSUPPORTED               # scales of fp32 states
    assert call(bits=16) == UNSUPPORTED
    assert call(dtypes=(BF16, 2)) == UNSUPPORTED
    for bad in (dict(count=0), dict(count=-1), dict(sizes=(300, 0)), dict(sizes=((1 << 33) + 1, 5)),
                dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=-1.0),
                dict(step=0), dict(count=(1 << 24) + 1)):
        assert call(**bad) == DIMS, bad
    for bad in (dict(p0=p["p0"] + 2), dict(g0=p["g0"] + 1), dict(g1=p["g1"] + 2), dict(c0=p["c0"] + 1),
                dict(m=p["m"] + 8), dict(ms=p["ms"] + 2)):
        assert call(ptrs=bad) == ALIGN, bad
    assert call(lr_value=BASE + 2) == ALIGN and call(step_value=BASE + 4) == ALIGN
    for bad in (dict(p1=p["p0"]),                          # the same tensor twice
                dict(p1=p["p0"] + 4 * 299), dict(c0=p["c1"] - 2 * 299), dict(p0=p["g1"]),
                dict(m=p["v"] + 256), dict(m=p["v"] - 384 - 112), dict(ms=p["g0"]),
                dict(vs=p["ms"] + 12)):                    # 300 and 5 are 4 blocks: 16 bytes
        assert call(ptrs=bad) == ALIAS, bad
    assert call(lr_value=p["p0"] + 8) == ALIAS
    assert call(bits=32, ptrs={**none, "m": p["v"] + 16 * 127}) == ALIAS
    # one gradient may serve two tensors: not an alias; the next refusal is reached
    assert call(ptrs=dict(g1=p["g0"]), dtypes=(F32, F32), lr_value=p["m"]) == ALIAS


def test_python_refuses_cpu_tensors():
    import torch
    import selective_state_space_52_amd as m
    x, t, f = torch.zeros(4, 128), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    state = m.adamw_state([x])
    for call in (lambda: m.embedding_fwd(t, x), lambda: m.embedding_bwd(t, x, 10),
                 lambda: m.token_logprobs_fwd(x, t),
                 lambda: m.token_logprobs_bwd(x, t, torch.zeros(4, 2), f),
                 lambda: m.policy_loss(x, t, f, f), lambda: m.preference_loss(f, f, off),
                 lambda: m.adamw_step([x], [x], state[0], state[1], step=1, lr=1e-3),
                 lambda: m.adamw_state([x], bits=16), lambda: m.adamw_state([])):
        with pytest.raises(ValueError):
            call()


def test_adamw_state_layout():
    import torch
    import selective_state_space_52_amd as mssm
    params = [torch.zeros(n) for n in (1, 128, 129)] + [torch.zeros(3, 100)]
    m, v, ms, vs = mssm.adamw_state(params)
    assert m.shape == v.shape == (128 * (1 + 1 + 2 + 3),) and ms is None and vs is None
    m, v, ms, vs = mssm.adamw_state(params, bits=8)
    assert m.dtype == v.dtype == torch.float8_e4m3fn and ms.shape == vs.shape == (7,)
    assert float(m.float().abs().max()) == 0.0 and float(ms.max()) == 0.0
