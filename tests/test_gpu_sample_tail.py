"""Sampling where many unlikely tokens together carry mass: what top_p keeps of
a long tail, against the definition in 64 bits."""
import math

import pytest
import torch

from tests import layer_common as lc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [50304, (1 << 21) + 5, 1 << 22])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tail_of_equal_tokens(vocab, dtype):
    """One token of w = 1 and a tail of equal ones of about 0.4 * 2^-31 each, 4e-4 in
    all for 2^21 of them.  With top_p in the middle of the tail's mass the first
    half of the tail (by index) stays: the tokens at its quarters, whose noise lets
    them win where the likely one's does not, tell which half is kept, and the
    log-probability how much of it."""
    import selective_state_space_52_amd as m
    logits = torch.full((2, vocab), math.log(0.4 * 2.0 ** -31)).to(dtype)
    logits[:, 3] = 0.0
    w = math.exp(float(logits[0, 0]))
    tail = (vocab - 1) * w
    noise = torch.full((2, vocab), 0.5)
    noise[1, 3] = 0.0
    noise[1, vocab // 4], noise[1, 3 * vocab // 4] = 1 - 2.0 ** -23, 1 - 2.0 ** -24
    top_p = (1 + tail / 2) / (1 + tail)
    tokens, lp = m.sample_tokens(logits.cuda(), noise.cuda(), top_p=top_p)
    kept = math.log1p(tail / 2)
    # masses: half a unit of 2^-41 a token; top_p, the sum and its logarithm in fp32:
    # 4 roundings of a number near 1; the scaled logit: 3 of its own
    slack = (vocab * 2.0 ** -42 + 8 * lc.U32) * (1 + tail)
    if tail > 1e-4:     # the middle of the tail is further than that from its quarters
        assert tokens.tolist() == [3, vocab // 4]
        assert abs(float(lp[1]) - (math.log(w) - kept)) <= slack + 4 * lc.U32 * abs(math.log(w))
    assert abs(float(lp[0]) + kept) <= slack + tail / 2 * (tail < 1e-4)
