"""The torch layers over the block operators on the GPU: EQLayerNorm and EQMLPBlock against the
fp64 oracle, against differences, and in the memory that a training step holds.

Bounds.  The outputs: the layer's own (1e-5 and 3e-3 of the norm), three products deep.  With
8-bit checkpoints the oracle rounds the same activations; where the two disagree on a code (their
inputs differ by err, a step is at most 1/64 of the block's largest value) they differ by one
step, so gradients may be off by sqrt(err / 64) of their norm: 1e-3 for err = 2e-6 (fp32) and
1.5e-2 for err = 1e-3 (fp16, some 2e-3 to 3e-3 each through four such roundings).  Against the unrounded gradient: half a step is at most
1/128 of the block's largest value, about three times its root mean square, so below 4%.
"""
import numpy as np
import pytest
import torch

from group_circulant_linear_p4_amd.layer import EQLayerNorm, EQMLPBlock, eq_layer_norm
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f16": torch.float16, "f32": torch.float32}


def rel(got, ref):
    got = got.detach().cpu().numpy().astype(np.float64)
    return float(np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30))


def make_block(c, h, t, dtype, ckpt8, seed=0):
    torch.manual_seed(seed)
    block = EQMLPBlock(c, h, t, device=DEV, dtype=DT[dtype], ckpt8=ckpt8)
    with torch.no_grad():
        block.norm.weight.add_(0.2 * torch.randn_like(block.norm.weight))
        for p in (block.norm.bias, block.fc1.bias, block.fc2.bias):
            p.add_(0.2 * torch.randn_like(p))
    return block


def params(block):
    return {"gamma": block.norm.weight, "beta": block.norm.bias, "w1": block.fc1.weight, "b1": block.fc1.bias,
            "w2": block.fc2.weight, "b2": block.fc2.bias}


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("ckpt8", [True, False])
@pytest.mark.parametrize("shape", [(3, 67, 24, 40, 4), (1, 300, 10, 25, 3), (2, 128, 16, 64, 8), (1, 1, 8, 8, 1)], ids=str)
def test_mlp_block(shape, ckpt8, dtype):
    b, n, c, h, t = shape
    print("case block", shape, ckpt8, dtype, flush=True)
    block = make_block(c, h, t, dtype, ckpt8)
    x = (torch.randn(b, n, c * t, device=DEV) * 1.5 + 0.3).to(DT[dtype]).requires_grad_(True)
    dy = torch.randn(b, n, c * t, device=DEV).to(DT[dtype])
    y = block(x)
    y.backward(dy)
    np64 = lambda v: v.detach().double().cpu().numpy()  # noqa: E731
    flat = lambda v: np64(v).reshape(b * n, c * t)  # noqa: E731
    ps = {k: np64(v) for k, v in params(block).items()}
    args = (flat(x), ps["gamma"], ps["beta"], ps["w1"], ps["b1"], ps["w2"], ps["b2"], 1e-5, flat(dy))
    ry, rg = B.mlp_block(*args, ckpt8)
    assert y.shape == x.shape and rel(y.reshape(b * n, -1), ry) <= (3e-5 if dtype == "f32" else 9e-3)
    got = {"x": x.grad.reshape(b * n, -1), **{k: v.grad for k, v in params(block).items()}}
    tol = (1e-3 if dtype == "f32" else 1.5e-2) if ckpt8 else (3e-5 if dtype == "f32" else 9e-3)
    for k, v in got.items():
        assert rel(v, rg[k]) <= tol, (k, rel(v, rg[k]))
    if ckpt8 and b * n > 100:
        _, plain = B.mlp_block(*args, False)
        for k, v in got.items():
            assert rel(v, plain[k]) <= 0.04, (k, rel(v, plain[k]))


def test_mlp_block_partial_gradients():
    """Every subset of parameters that a caller freezes leaves the others' gradients as they were."""
    x = torch.randn(50, 32, device=DEV).half()
    dy = torch.randn(50, 32, device=DEV).half()

    def grads(wanted, need_x):
        block = make_block(8, 12, 4, "f16", True)
        for k, p in params(block).items():
            p.requires_grad_(k in wanted)
        xi = x.clone().requires_grad_(need_x)
        block(xi).backward(dy)
        return {**{k: p.grad for k, p in params(block).items()}, "x": xi.grad}

    names = ["gamma", "beta", "w1", "b1", "w2", "b2"]
    full = grads(names, True)
    for wanted, need_x in ((["w2"], False), (["b2"], False), (["b1"], False), (["w1"], False), (["gamma"], False),
                           ([], True), (["w1", "w2"], False), (["beta", "b1"], True)):
        got = grads(wanted, need_x)
        for k in names + ["x"]:
            if k in wanted or (k == "x" and need_x):
                # A weight gradient alone takes dy's spectrum from another kernel: one rounding apart.
                assert rel(got[k].float(), full[k].double().cpu().numpy()) <= 2e-3, (wanted, k)
            else:
                assert got[k] is None, (wanted, k)


def test_mlp_block_holds_less_memory_and_no_graph_without_grad():
    n, c, h, t = 4096, 64, 256, 4
    x = torch.randn(n, c * t, device=DEV).half()

    def held(ckpt8):
        block = make_block(c, h, t, "f16", ckpt8)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y = block(x)
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated() - before - y.numel() * 2

    small, large = held(True), held(False)
    # C' + H' bytes per group element and row, a scale byte for 32, and 1 / std.
    want = n * t * (c + h)
    assert want <= small <= 1.05 * want + (1 << 20) and large >= 4 * small
    with torch.no_grad():
        block = make_block(c, h, t, "f16", True)
        y = block(x)
        assert not y.requires_grad
    assert torch.equal(y, block(x.clone().requires_grad_(True)).detach())


def test_mlp_block_is_equivariant():
    """A cyclic shift of every channel's group axis goes through the block, in 64-bit differences
    of the outputs' rounding only."""
    c, h, t = 16, 32, 4
    block = make_block(c, h, t, "f32", True)
    x = torch.randn(40, c * t, device=DEV)
    shift = lambda v: torch.roll(v.reshape(-1, c, t), 1, 2).reshape(-1, c * t)  # noqa: E731
    a, b = block(shift(x)), shift(block(x))
    assert rel(a, b.detach().double().cpu().numpy()) <= 1e-5


@pytest.mark.parametrize("ckpt8", [False, True])
def test_layer_norm_layer_and_differences(ckpt8):
    c, t = 20, 3
    norm = EQLayerNorm(c, t, device=DEV, dtype=torch.float32, ckpt8=ckpt8)
    with torch.no_grad():
        norm.weight.uniform_(0.5, 1.5)
        norm.bias.normal_()
    x = torch.randn(4, 9, c * t, device=DEV, requires_grad=True)
    dy, v = torch.randn_like(x), torch.randn_like(x)
    norm(x).backward(dy)
    with torch.no_grad():
        step = 1e-2
        diff = ((norm(x + step * v).double() - norm(x - step * v).double()) * dy.double()).sum() / (2 * step)
        got = (x.grad.double() * v.double()).sum()
        # Differences: third derivative times step^2 / 6 and fp32 rounding over the step; 8 bits: 4%
        # of the gradient's norm along v.
        slack = 1e-3 * (x.grad.norm() * v.norm()).item() + (0.04 * x.grad.norm().item() if ckpt8 else 0.0)
        assert abs((diff - got).item()) <= slack
    y, h, _, rstd = B.norm(x.detach().cpu().numpy().reshape(36, -1), norm.weight.detach().cpu().numpy(),
                           norm.bias.detach().cpu().numpy(), t, 1e-5)
    if ckpt8:
        h = B.unpack(*B.pack(h), c * t)
    dx, dg, db = B.norm_bwd(dy.cpu().numpy().reshape(36, -1), h, rstd, norm.weight.detach().cpu().numpy(), t)
    tol = 1e-3 if ckpt8 else 1e-5
    assert rel(norm(x).reshape(36, -1), y) <= 1e-5 and rel(x.grad.reshape(36, -1), dx) <= tol
    assert rel(norm.weight.grad, dg) <= tol and rel(norm.bias.grad, db) <= 1e-5


def test_layer_norm_layer_takes_strided_and_empty_inputs():
    x = torch.randn(6, 10, 24, device=DEV).half()
    strided = x.transpose(0, 1)[::2]
    want = eq_layer_norm(strided.contiguous(), group_order=4)
    assert torch.equal(eq_layer_norm(strided, group_order=4), want) and want.shape == strided.shape
    empty = torch.empty(0, 24, device=DEV, dtype=torch.float16, requires_grad=True)
    norm = EQLayerNorm(6, 4, device=DEV, dtype=torch.float16, ckpt8=True)
    norm(empty).sum().backward()
    assert empty.grad.shape == (0, 24) and not norm.weight.grad.any().item()
    block = EQMLPBlock(6, 8, 4, device=DEV, dtype=torch.float16)
    block(empty).sum().backward()
    assert all(not p.grad.any().item() for p in block.parameters())


def test_example_trains():
    import argparse
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block.py")
    spec = importlib.util.spec_from_file_location("mlp_block_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    a = argparse.Namespace(rows=512, channels=12, hidden=24, group=4, steps=30, rate=0.3, dtype="f16")
    losses = [example.train(a, ckpt8) for ckpt8 in (True, False)]
    assert all(last < 0.7 * first for first, last in losses)
    # The same task with rounded and whole activations: the same descent to a few per cent.
    assert abs(losses[0][1] - losses[1][1]) <= 0.04 * losses[1][1]


@pytest.mark.parametrize("ckpt8", [False, True])
def test_mlp_block_gradient_against_differences(ckpt8):
    """Directional derivatives of the block in x and in every parameter, fp32: central differences
    (error: third derivative times step^2 / 6 and fp32 rounding of the outputs over the step, 2e-3
    of the product of norms), and 4% of the gradient's norm along the direction with 8 bits."""
    block = make_block(12, 20, 4, "f32", ckpt8, seed=5)
    x = torch.randn(64, 48, device=DEV, requires_grad=True)
    dy = torch.randn(64, 48, device=DEV)
    block(x).backward(dy)
    step = 1e-2
    for name, p in [("x", x), *params(block).items()]:
        v = torch.randn_like(p)
        v /= v.norm()
        with torch.no_grad():
            p.add_(step * v)
            hi = (block(x).double() * dy.double()).sum()
            p.sub_(2 * step * v)
            lo = (block(x).double() * dy.double()).sum()
            p.add_(step * v)
        got = (p.grad.double() * v.double()).sum().item()
        slack = (0.04 if ckpt8 else 2e-3) * p.grad.norm().item() + 2e-3 * dy.norm().item()
        assert abs(((hi - lo) / (2 * step)).item() - got) <= slack, name


def test_default_stream_argument_is_torchs_current_stream():
    import group_circulant_linear_p4_amd as eql
    torch.cuda.init()
    assert (eql._stream(None) or 0) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert eql._stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
    assert (eql._stream(None) or 0) == torch.cuda.current_stream().cuda_stream


def test_layers_take_slices_off_a_16_byte_boundary():
    """Rows of 15 fp16 features: a slice from row 1 on starts 30 bytes into its tensor, and so does
    the gradient that torch.cat's backward hands to the second of two."""
    torch.manual_seed(4)
    norm = EQLayerNorm(5, 3, device=DEV, dtype=torch.float16)
    block = make_block(5, 7, 3, "f16", True)
    whole = torch.randn(9, 15, device=DEV, dtype=torch.float16)
    dy = torch.randn(9, 15, device=DEV, dtype=torch.float16)
    for f in (norm, block):
        grads = []
        for part, start in ((whole[1:], 14), (whole[1:].clone(), 0)):
            x = part.detach().requires_grad_(True)
            assert x.data_ptr() % 16 == start
            f.zero_grad()
            torch.cat([whole[:1], f(x)]).backward(dy)
            grads.append([x.grad] + [p.grad.clone() for p in f.parameters()])
        assert all(torch.equal(a, b) for a, b in zip(*grads))
