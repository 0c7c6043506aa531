"""The settings that sample_tokens hands to the library, on the CPU (nothing is
launched)."""
import pytest
import torch


@pytest.mark.parametrize("top_k,want", [(5, 5), (0, 0), (-1, 0), (2**31 - 1, 2**31 - 1), (2**31, 2**31 - 1),
                                        (2**32 + 5, 2**31 - 1), (-2**31, 0), (5 - 2**32, 0), (1 - 2**33, 0)])
def test_top_k(monkeypatch, top_k, want):
    """Any integer: <= 0 is all tokens, what exceeds 32 bits more than any row has."""
    from selective_state_space_52_amd import layer
    got = []
    monkeypatch.setattr(layer, "_io", lambda t, name, dims: 0)
    monkeypatch.setattr(layer, "_call", lambda device, fn, *args: got.append(args[-1].top_k))
    x = torch.zeros(2, 7)
    layer.sample_tokens(x, x, top_k=top_k)
    assert got == [want]
