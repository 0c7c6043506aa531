"""Limits of the ends of a training step that validation holds, and that the Python
calls know as numbers of their own; nothing here reaches a GPU."""
import pytest

from tests.test_layer_abi import DIMS, far
from tests.test_train_abi import L, _logp, _policy  # noqa: F401


@pytest.mark.parametrize("t", [1e-45, 2.9e-39, 3.5e-39, 4.2e-39])
def test_temperatures_too_small_to_divide_by(L, t):  # noqa: F811
    """log2(e) / t has to be finite: 0 times it, the largest logit's exponent, would
    be NaN otherwise.  The smallest t is 4.24e-39."""
    p = far(("logits", "tokens", "logprobs", "stats", "old", "adv", "loss", "dlogits", "d"))
    at = p.get
    assert L.mssm_token_logprobs_fwd(at("logits"), at("tokens"), at("logprobs"), at("stats"), None, 0,
                                     _logp(t=t), None) == DIMS
    assert L.mssm_token_logprobs_bwd(at("logits"), at("tokens"), at("stats"), at("d"), at("dlogits"),
                                     _logp(t=t), None) == DIMS
    assert L.mssm_policy_loss(at("logits"), at("tokens"), at("old"), at("adv"), None, None, at("loss"),
                              at("logprobs"), at("dlogits"), None, 0, _policy(t=t), None) == DIMS


def test_limits_that_python_knows(L):  # noqa: F811
    """train.py asks for no workspace up to these sizes: they are the kernels' own."""
    import ctypes
    from selective_state_space_52_amd import train
    from tests.test_train_abi import _embed
    n = ctypes.c_int64(-1)
    for size, call, dims in ((train._UNSORTED, L.mssm_embedding_bwd_workspace, lambda k: _embed(rows=k)),
                             (train._WHOLE, L.mssm_token_logprobs_workspace, lambda k: _logp(vocab=k))):
        assert call(dims(size), n) == 0 and n.value == 0
        assert call(dims(size + 1), n) == 0 and n.value > 0


def test_no_states_for_an_empty_tensor():
    """adamw_step refuses it, so its states are refused too."""
    import torch
    import selective_state_space_52_amd as m
    for bits in (32, 8):
        with pytest.raises(ValueError):
            m.adamw_state([torch.zeros(3), torch.zeros(0, 4)], bits)
