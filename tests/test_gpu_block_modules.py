"""The torch layers as modules, on the GPU."""
import pytest
import torch

from group_circulant_linear_p4_amd.layer import EQLayerNorm, EQLinear, EQLinearP4M, EQMLPBlock

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16 = torch.float16


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


def off_boundary(p):
    """The parameter's values, two bytes past a 16-byte boundary."""
    room = torch.empty(p.numel() + 1, dtype=p.dtype, device=p.device)
    room[1:] = p.detach().reshape(-1)
    return torch.nn.Parameter(room[1:].view(p.shape))


LAYERS = {
    "block": (15, lambda: EQMLPBlock(5, 7, 3, device=DEV, dtype=F16, ckpt8=True)),
    "block whole": (15, lambda: EQMLPBlock(5, 7, 3, device=DEV, dtype=F16, ckpt8=False)),
    "linear": (15, lambda: EQLinear(5, 7, 3, device=DEV, dtype=F16)),
    "linear no spectra": (15, lambda: EQLinear(5, 7, 3, device=DEV, dtype=F16, keep_spectra=False)),
    "linear fused": (15, lambda: EQLinear(5, 7, 3, bias=True, activation="gelu", device=DEV, dtype=F16)),
    "p4m": (8, lambda: EQLinearP4M(1, 3, device=DEV, dtype=F16)),
}


@pytest.mark.parametrize("weights", ["as made", "off the boundary"])
@pytest.mark.parametrize("name", list(LAYERS))
def test_layers_take_any_contiguous_slice(name, weights):
    """Rows from the second feature on of a flat tensor, weights likewise (as in a flattened parameter
    buffer), and the gradient that torch.cat's backward hands out: as from aligned copies."""
    features, make = LAYERS[name]
    torch.manual_seed(4)
    f = make()
    flat = torch.randn(8 * features + 1, device=DEV, dtype=F16)
    want = None
    for aligned in (True, False):
        x = flat[1:].view(8, features).detach()
        x = (x.clone() if aligned else x).requires_grad_(True)
        assert x.data_ptr() % 16 == (0 if aligned else 2)
        if weights != "as made" and not aligned:
            for m in f.modules():
                for k, p in list(m.named_parameters(recurse=False)):
                    setattr(m, k, off_boundary(p))
        f.zero_grad()
        y = f(x)
        torch.manual_seed(9)
        dy = torch.randn(1 + y.numel(), device=DEV, dtype=F16)
        torch.cat([dy[:1], y.reshape(-1)]).backward(dy)
        got = [y.detach(), x.grad] + [p.grad for p in f.parameters()]
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        want = [v.clone() for v in got]


def test_fused_layer_takes_a_residual_off_the_boundary():
    torch.manual_seed(5)
    f = EQLinear(5, 5, 3, device=DEV, dtype=F16)
    x, flat = torch.randn(8, 15, device=DEV, dtype=F16), torch.randn(8 * 15 + 1, device=DEV, dtype=F16)
    r = flat[1:].view(8, 15)
    assert torch.equal(f(x, r), f(x, r.clone()))


@pytest.mark.parametrize("make", [lambda: EQLayerNorm(6, 4, device=DEV), lambda: EQLayerNorm(6, 4, device=DEV, ckpt8=True),
                                  lambda: EQMLPBlock(6, 10, 4, device=DEV), lambda: EQMLPBlock(6, 10, 4, device=DEV, ckpt8=False),
                                  lambda: EQLinear(6, 10, 4, device=DEV), lambda: EQLinear(6, 10, 4, bias=True, device=DEV),
                                  lambda: EQLinearP4M(3, 5, device=DEV)],
                         ids=["norm", "norm 8bit", "block 8bit", "block", "linear", "linear fused", "p4m"])
def test_gradients_of_gradients_are_refused(make):
    """The backward passes have no derivative of their own: asking for one raises, where a gradient
    without a graph would count as a constant."""
    torch.manual_seed(1)
    f = make()
    x = torch.randn(7, 24, device=DEV, requires_grad=True)
    first, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    plain, = torch.autograd.grad(f(x).square().sum(), x)
    assert torch.equal(first.detach(), plain)
    # Beside a term that has its second derivative, as a penalty on the gradient's norm would be.
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (first.square().sum() + x.square().sum()).backward()


def along(fn, p, v, dy, eps):
    """Central difference of sum(fn() dy) in p along v."""
    with torch.no_grad():
        p.add_(eps * v)
        hi = (fn().double() * dy.double()).sum()
        p.sub_(2 * eps * v)
        lo = (fn().double() * dy.double()).sum()
        p.add_(eps * v)
    return ((hi - lo) / (2 * eps)).item()


@pytest.mark.parametrize("ckpt8", [False, True])
def test_block_gradients_along_their_own_direction(ckpt8):
    """Along v = grad / |grad| the derivative is |grad| where the gradient is right (along a random
    direction it is some |grad| / sqrt(size), less than what rounding to 8 bits may cost).  Central
    differences with a step of 1e-2: the outputs' fp32 rounding, 2^-24 |y| an element, weighted by dy
    and over twice the step, below 1e-3; the third derivative times step^2 / 6, below 1e-3 of |grad|:
    1% of |grad|, which is 10 or more here, holds both.  8 bits: 4% more.  A gradient of zeros, one of
    the other sign, one of half the size and a random one of the same length are all outside."""
    torch.manual_seed(5)
    block = EQMLPBlock(12, 20, 4, device=DEV, ckpt8=ckpt8)
    with torch.no_grad():
        block.norm.weight.add_(0.2 * torch.randn_like(block.norm.weight))
        for p in (block.norm.bias, block.fc1.bias, block.fc2.bias):
            p.add_(0.2 * torch.randn_like(p))
    x = torch.randn(64, 48, device=DEV, requires_grad=True)
    dy = torch.randn(64, 48, device=DEV)
    block(x).backward(dy)
    tol = 0.05 if ckpt8 else 0.01
    for name, p in [("x", x), *block.named_parameters()]:
        grad, rand = p.grad, torch.randn_like(p)
        fits = []
        for claim in (grad, torch.zeros_like(grad), -grad, 0.5 * grad, rand * (grad.norm() / rand.norm())):
            v = grad / grad.norm()
            diff = along(lambda: block(x), p, v, dy, 1e-2)
            fits.append(abs(diff - (claim.double() * v.double()).sum().item()) <= tol * abs(diff))
        assert fits == [True, False, False, False, False], (name, fits)
