"""What the differentiable feed-forward block keeps for a backward: nothing where none can come."""

import pytest
import torch


@pytest.fixture
def saves(monkeypatch):
    """The ``save`` of each forward that the block makes (the call itself replaced: no GPU here)."""
    from matrix_orthogonalising_optimizer_muon_amd import layers
    seen = []

    def forward(x, w_gate, w_up, w_down, *, activation="silu", save=False):
        seen.append(save)
        return x * 2.0, torch.zeros(1) if save else None
    monkeypatch.setattr(layers, "ffn_forward", forward)
    return layers, seen


def test_block_saves_only_for_a_backward_that_can_come(saves):
    layers, seen = saves
    block = layers.GatedFeedForward(4, 6, dtype=torch.float32)
    x = torch.zeros(3, 4)
    assert block(x).requires_grad
    with torch.no_grad():
        assert not block(x).requires_grad
    with torch.inference_mode():
        block(x)
    for p in block.parameters():
        p.requires_grad_(False)
    assert not block(x).requires_grad
    assert block(x.requires_grad_(True)).requires_grad
    assert seen == [True, False, False, False, True]
