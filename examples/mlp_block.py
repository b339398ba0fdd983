"""Trains one pre-norm EQ-Linear MLP block on synthetic data, with its activations kept in 8 bits
and with them kept whole, and prints the loss, the time of a step and the memory that a block holds
from its forward to its backward pass.

    python examples/mlp_block.py [--rows N] [--channels C] [--hidden H] [--group T] [--steps K] [--dtype f16|f32]

The task: match another block's outputs on random rows.  Needs an MI355X and the built library.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from group_circulant_linear_p4_amd.layer import EQMLPBlock  # noqa: E402


def train(a, ckpt8: bool):
    """The first and the last step's loss."""
    dtype = torch.float16 if a.dtype == "f16" else torch.float32
    torch.manual_seed(0)
    teacher = EQMLPBlock(a.channels, a.hidden, a.group, device="cuda", dtype=dtype)
    block = EQMLPBlock(a.channels, a.hidden, a.group, device="cuda", dtype=dtype, ckpt8=ckpt8)
    x = torch.randn(a.rows, a.channels * a.group, device="cuda", dtype=dtype)
    with torch.no_grad():
        target = teacher(x)
    # fp32 master weights; the block computes on their rounded copies.
    master = [p.detach().float() for p in block.parameters()]
    moments = [torch.zeros_like(m) for m in master]
    losses, held, began = [], 0, 0.0
    for step in range(a.steps + 3):
        if step == 3:
            torch.cuda.synchronize()
            began = time.perf_counter()
        y = diff = None
        before = torch.cuda.memory_allocated()
        y = block(x)
        held = torch.cuda.memory_allocated() - before - y.numel() * y.element_size()
        diff = (y - target).float()
        losses.append(diff.square().mean())
        # The loss is a sum over rows here, so that fp16 gradients stay in range.
        y.backward((2.0 * diff / a.rows ** 0.5).to(dtype))
        with torch.no_grad():
            for p, m, v in zip(block.parameters(), master, moments):
                g = p.grad.float() / (a.rows ** 0.5 * diff.shape[1])
                v.mul_(0.9).add_(g)
                m.add_(v, alpha=-a.rate)
                p.copy_(m)
                p.grad = None
    torch.cuda.synchronize()
    ms = (time.perf_counter() - began) / a.steps * 1e3
    print("%-22s loss %.5f -> %.5f   %.3f ms a step   %.1f MB held by the block" % (
        "8-bit activations:" if ckpt8 else "whole activations:", losses[0].item(), losses[-1].item(), ms, held / 1e6), flush=True)
    return losses[0].item(), losses[-1].item()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=12608)
    ap.add_argument("--channels", type=int, default=96)
    ap.add_argument("--hidden", type=int, default=384)
    ap.add_argument("--group", type=int, default=4)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--rate", type=float, default=0.3)
    ap.add_argument("--dtype", choices=("f16", "f32"), default="f16")
    a = ap.parse_args()
    for ckpt8 in (True, False):
        train(a, ckpt8)


if __name__ == "__main__":
    main()
