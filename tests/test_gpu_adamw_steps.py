"""The AdamW step where it repeats itself or its numbers are at their type's ends."""
import pytest
import torch

from tests import layer_common as lc

pytestmark = pytest.mark.gpu
U32 = lc.U32


def states(mssm, params, bits):
    m, v, ms, vs = mssm.adamw_state(params, bits)
    return (m, v), dict(m_scales=ms, v_scales=vs)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-20, 1e-8])
def test_squares_below_the_normal_numbers(bits, eps):
    """Gradients of 1e-19: v is 1e-41, whose root is 3e-21.  The step is lr g / (|g| +
    eps) with it, and neither lr g / eps nor an infinity.

    The square, 1e-38, and v are each rounded to a multiple of 2^-149, so v is off by
    2^-150 (1 + 1e-3), the step by half of that relative to v, and 8 roundings."""
    import selective_state_space_52_amd as mssm
    g = torch.full((300,), 1e-19, device="cuda")
    g[1::2] *= -1
    g[5], g[200] = 0.5, -2.0                    # beside ordinary ones
    p = torch.ones(300, device="cuda")
    mv, scales = states(mssm, [p], bits)
    mssm.adamw_step([p], [g], *mv, step=1, lr=0.1, eps=eps, weight_decay=0.0, **scales)
    gd = g.double().cpu()
    want = 1.0 - 0.1 * gd / (gd.abs() + eps)
    off = 0.1 * (2.0 ** -150 * 1.001 / 1e-41 / 2 + 8 * U32)
    assert float((p.double().cpu() - want).abs().max()) <= off + U32
