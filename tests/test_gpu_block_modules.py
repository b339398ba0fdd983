"""The torch layers as modules, on the GPU."""
import pytest
import torch

from group_circulant_linear_p4_amd.layer import EQLinear, EQMLPBlock

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def step(block, x, dy):
    """The output and the gradients by name."""
    x = x.clone().requires_grad_(True)
    block.zero_grad()
    y = block(x)
    y.backward(dy)
    return {"y": y.detach(), "x": x.grad, **{k: p.grad.clone() for k, p in block.named_parameters() if p.grad is not None}}


def close(got, want, tol):
    return all((got[k].double() - want[k].double()).norm() <= tol * want[k].double().norm() + 1e-12 for k in want)


def composed(block, x, dy):
    """The same step through the submodules, one after the other."""
    plain = lambda v: block.fc2(block.fc1(block.norm(v)), residual=v)  # noqa: E731
    x = x.clone().requires_grad_(True)
    block.zero_grad()
    y = plain(x)
    y.backward(dy)
    return {"y": y.detach(), "x": x.grad, **{k: p.grad.clone() for k, p in block.named_parameters() if p.grad is not None}}


def changes():
    def hook(b):
        b.fc1.register_forward_hook(lambda m, i, o: 2.0 * o)

    def pre_hook(b):
        # A weight recomputed before each call, as weight normalisation does.
        def recompute(m, inputs):
            m.weight.data.fill_(0.1)
        b.fc2.register_forward_pre_hook(recompute)

    def activation(b):
        b.fc1.activation = None

    def own_forward(b):
        b.norm.forward = lambda v: 0.5 * v

    def identity(b):
        b.norm = torch.nn.Identity()

    def no_bias(b):
        b.fc1.bias = None

    def subclass(b):
        class Scaled(EQLinear):
            def forward(self, x, residual=None):
                return super().forward(3.0 * x, residual)
        old, b.fc2 = b.fc2, Scaled(20, 12, 4, bias=True, device=DEV)
        b.fc2.load_state_dict(old.state_dict())

    return [hook, pre_hook, activation, own_forward, identity, no_bias, subclass]


@pytest.mark.parametrize("change", changes(), ids=lambda f: f.__name__)
def test_block_follows_its_submodules(change):
    """What a user hooks into, replaces in or sets on norm, fc1 and fc2 takes effect with 8-bit
    activations as it does without."""
    torch.manual_seed(6)
    block = EQMLPBlock(12, 20, 4, device=DEV)
    with torch.no_grad():
        block.fc1.bias.add_(1.0)
    x, dy = torch.randn(40, 48, device=DEV), torch.randn(40, 48, device=DEV)
    before = block(x).detach()
    change(block)
    got, want = step(block, x, dy), composed(block, x, dy)
    assert (before - want["y"]).norm() > 0.01 * want["y"].norm()  # the change matters
    assert close(got, want, 1e-5)


def test_block_runs_hooks_and_keeps_8_bits_without_them():
    torch.manual_seed(7)
    block = EQMLPBlock(12, 20, 4, device=DEV)
    x, dy = torch.randn(40, 48, device=DEV), torch.randn(40, 48, device=DEV)
    plain = step(block, x, dy)
    seen = []
    handles = [m.register_forward_hook(lambda m, i, o: seen.append(type(m).__name__)) for m in (block.norm, block.fc1, block.fc2)]
    block(x)
    assert seen == ["EQLayerNorm", "EQLinear", "EQLinear"]
    for h in handles:
        h.remove()
    again = step(block, x, dy)
    assert seen == ["EQLayerNorm", "EQLinear", "EQLinear"] and all(torch.equal(plain[k], again[k]) for k in plain)
    # Whole activations give other gradients: those above came from the 8-bit ones.
    assert not torch.equal(plain["fc2.weight"], composed(block, x, dy)["fc2.weight"])


def test_block_with_a_parametrised_weight_keeps_8_bits():
    """A parametrisation changes the value of the attribute, which both ways read."""
    class Double(torch.nn.Module):
        def forward(self, w):
            return 2.0 * w

    torch.manual_seed(8)
    block, same = EQMLPBlock(12, 20, 4, device=DEV), EQMLPBlock(12, 20, 4, device=DEV)
    same.load_state_dict(block.state_dict())
    with torch.no_grad():
        same.fc1.weight.mul_(2.0)
    torch.nn.utils.parametrize.register_parametrization(block.fc1, "weight", Double())
    x, dy = torch.randn(40, 48, device=DEV), torch.randn(40, 48, device=DEV)
    a, b = step(block, x, dy), step(same, x, dy)
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["x"], b["x"]) and torch.equal(a["fc2.weight"], b["fc2.weight"])
    assert torch.equal(block.fc1.parametrizations.weight.original.grad, 2.0 * same.fc1.weight.grad)


def test_block_runs_hooks_on_all_modules():
    block = EQMLPBlock(12, 20, 4, device=DEV)
    seen = []
    handle = torch.nn.modules.module.register_module_forward_hook(lambda m, i, o: seen.append(type(m).__name__))
    try:
        block(torch.randn(4, 48, device=DEV))
    finally:
        handle.remove()
    assert seen == ["EQLayerNorm", "EQLinear", "EQLinear", "EQMLPBlock"]
