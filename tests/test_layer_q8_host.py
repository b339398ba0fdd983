"""What the 8-bit torch layers decide on the host: which modules they take, and which gradients they refuse (no GPU
needed: modules that compute on the CPU stand in for the layers).
"""
import pytest
import torch

from group_circulant_linear_p4_amd import layer


class Doubled(torch.nn.Module):
    """In an 8-bit layer's place: 2 x + residual, without parameters."""

    def forward(self, x, residual=None):
        return 2 * x if residual is None else 2 * x + residual


def test_a_block_with_a_trained_norm_refuses_the_backward_pass():
    block = layer.EQMLPBlock8bit(torch.nn.LayerNorm(6), Doubled(), Doubled())
    x = torch.randn(3, 6)
    y = block(x)
    assert y.shape == x.shape and torch.equal(y, 4 * block.norm(x) + x)
    other = torch.ones(6, requires_grad=True)  # a loss that has other gradients
    with pytest.raises(RuntimeError, match="backward"):
        (y * other).sum().backward()
    assert block.norm.weight.grad is None
    with torch.no_grad():
        assert not block(x).requires_grad
    with pytest.raises(RuntimeError):
        block(x.requires_grad_(True))
    block.norm.requires_grad_(False)
    y = block(x.detach())
    assert not y.requires_grad
