"""What the 8-bit torch layers decide on the host: which modules they take, and which gradients they refuse (no GPU
needed: modules that compute on the CPU stand in for the layers).
"""
import pytest
import torch

from group_circulant_linear_p4_amd import layer


class Doubled(torch.nn.Module):
    """In an 8-bit layer's place: 2 x + residual, without parameters."""

    def forward(self, x, residual=None):
        return 2 * x if residual is None else (2 * x + residual).reshape(x.shape)


def test_a_block_with_a_trained_norm_refuses_the_backward_pass():
    block = layer.EQMLPBlock8bit(torch.nn.LayerNorm(6), Doubled(), Doubled())
    x = torch.randn(3, 6)
    y = block(x)
    assert y.shape == x.shape and torch.equal(y, 4 * block.norm(x) + x)
    other = torch.ones(6, requires_grad=True)  # a loss that has other gradients
    with pytest.raises(RuntimeError, match="backward"):
        (y * other).sum().backward()
    assert block.norm.weight.grad is None
    y = block(x)
    y += 1  # in place, also where fc2 returns a view
    with pytest.raises(RuntimeError, match="backward"):
        (y * other).sum().backward()
    with torch.no_grad():
        assert not block(x).requires_grad
    with pytest.raises(RuntimeError):
        block(x.requires_grad_(True))
    block.norm.requires_grad_(False)
    y = block(x.detach())
    assert not y.requires_grad


@pytest.fixture
def packed(monkeypatch):
    """Weights handed to the packing launch."""
    seen = []
    monkeypatch.setattr(layer, "eqlinear_q8_pack_weight", lambda w, *a: seen.append(w))
    monkeypatch.setattr(layer, "eqlinear_p4m_expand_weight", lambda *a: None)
    return seen


class Scaled(layer.EQLinear):
    def forward(self, x, residual=None):
        return 3 * super().forward(x, residual)


class Renamed(layer.EQLinear):
    """Computes what EQLinear does."""


def test_from_float_takes_what_it_can_keep(packed):
    for made in (layer.EQLinear(4, 6, 4, bias=True, activation="gelu"), Renamed(4, 6, 4), layer.EQLinearP4M(4, 6)):
        q = layer.EQLinear8bit.from_float(made)
        assert isinstance(q, layer.EQLinear8bit) and (q.bias is None) == (getattr(made, "bias", None) is None)
    assert len(packed) == 3
    for norm in ("layer", "rms"):
        block = layer.EQMLPBlock(4, 6, 4, norm=norm)
        q = layer.EQMLPBlock8bit.from_float(block)
        assert q.norm is block.norm and q.fc1.activation == "gelu"


def test_from_float_refuses_hooks_and_other_forwards(packed):
    def hooked(register):
        made = layer.EQLinear(4, 6, 4)
        getattr(made, register)(lambda *a: None)
        return made
    patched, p4m = layer.EQLinear(4, 6, 4), layer.EQLinearP4M(4, 6)
    patched.forward = lambda x, residual=None: x
    p4m.register_forward_hook(lambda *a: None)
    for bad in (Scaled(4, 6, 4), hooked("register_forward_hook"), hooked("register_forward_pre_hook"),
                hooked("register_full_backward_hook"), patched, p4m):
        with pytest.raises(ValueError):
            layer.EQLinear8bit.from_float(bad)
    block = layer.EQMLPBlock(4, 6, 4)
    block.fc2.register_forward_hook(lambda *a: None)
    with pytest.raises(ValueError):
        layer.EQMLPBlock8bit.from_float(block)
    block = layer.EQMLPBlock(4, 6, 4)
    block.register_forward_hook(lambda *a: None)
    with pytest.raises(ValueError):
        layer.EQMLPBlock8bit.from_float(block)

    class Other(layer.EQMLPBlock):
        def forward(self, x):
            return x - super().forward(x)
    with pytest.raises(ValueError):
        layer.EQMLPBlock8bit.from_float(Other(4, 6, 4))
    with pytest.raises(TypeError):
        layer.EQMLPBlock8bit.from_float(torch.nn.Sequential())
    with pytest.raises(TypeError):
        layer.EQLinear8bit.from_float(torch.nn.Linear(4, 4))
    assert not packed


def test_a_state_of_other_sizes_is_refused():
    """A packed weight is bytes: 12 outputs of 8 inputs take as many as 8 of 12, or as 30 of 20."""
    made = layer.EQLinear8bit(8, 12, 4)
    made.weight8.random_(0, 255)
    state = made.state_dict()
    again = layer.EQLinear8bit(8, 12, 4)
    again.load_state_dict(state)
    assert torch.equal(again.weight8, made.weight8)
    for sizes in ((12, 8, 4), (20, 30, 4)):
        other = layer.EQLinear8bit(*sizes)
        assert other.weight8.numel() == made.weight8.numel()
        for strict in (True, False):
            with pytest.raises(RuntimeError, match="channels"):
                other.load_state_dict(state, strict=strict)
        assert not other.weight8.any()
    # Within a model, under a prefix; a state saved without the sizes is taken as it was.
    model = torch.nn.Sequential(layer.EQLinear8bit(8, 12, 4), layer.EQLinear8bit(12, 8, 4))
    model.load_state_dict(model.state_dict())
    with pytest.raises(RuntimeError):
        torch.nn.Sequential(layer.EQLinear8bit(12, 8, 4), layer.EQLinear8bit(8, 12, 4)).load_state_dict(model.state_dict())
    again.load_state_dict({"weight8": made.weight8})
