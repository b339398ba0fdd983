"""CPU pins of the block operators' oracle (oracle/block_oracle.py): the norm's and the
checkpointed passes' gradients against central differences, torch's own layer norm at T = 1, the
equivariance the operators must keep, and the checkpoint format's properties."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block_oracle as B


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("n,c,t", [(3, 5, 1), (2, 4, 4), (4, 3, 3), (1, 2, 8)])
def test_norm_matches_torch_and_commutes_with_the_group(n, c, t):
    g = rng(n + c + t)
    x = g.standard_normal((n, c * t)) * 3 + 1
    gamma, beta = g.standard_normal(c), g.standard_normal(c)
    y, h, mean, rstd = B.norm(x, gamma, beta, t, 1e-5)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (c * t,), torch.from_numpy(np.repeat(gamma, t)),
                                         torch.from_numpy(np.repeat(beta, t)), 1e-5)
    assert np.allclose(y, ref.numpy(), rtol=0, atol=1e-12)
    shift = lambda v: np.roll(v.reshape(n, c, t), 1, axis=2).reshape(n, c * t)  # noqa: E731
    assert np.allclose(B.norm(shift(x), gamma, beta, t, 1e-5)[0], shift(y), rtol=0, atol=1e-13)


@pytest.mark.parametrize("n,c,t", [(3, 5, 1), (2, 4, 4), (4, 3, 3)])
def test_norm_gradients_match_differences(n, c, t):
    g = rng(10 + n)
    x, dy, dres = (g.standard_normal((n, c * t)) for _ in range(3))
    gamma, beta = g.standard_normal(c), g.standard_normal(c)
    loss = lambda x_, g_, b_: float((B.norm(x_, g_, b_, t, 1e-5)[0] * dy).sum() + (x_ * dres).sum())  # noqa: E731
    _, h, _, rstd = B.norm(x, gamma, beta, t, 1e-5)
    dx, dg, db = B.norm_bwd(dy, h, rstd, gamma, t, dres)
    step = 1e-5
    for grad, args in ((dx, 0), (dg, 1), (db, 2)):
        v = g.standard_normal(grad.shape)
        at = [x, gamma, beta]
        hi, lo = list(at), list(at)
        hi[args], lo[args] = at[args] + step * v, at[args] - step * v
        diff = (loss(*hi) - loss(*lo)) / (2 * step)
        assert abs(diff - float((grad * v).sum())) <= 1e-7 * max(1.0, abs(diff))


def test_gelu_and_weight_gradients_match_differences():
    g = rng(4)
    n, c, d, t = 5, 3, 4, 3
    pre, dy = g.standard_normal((n, d * t)), g.standard_normal((n, d * t))
    dpre, dbias = B.gelu_bwd(dy, pre, t)
    v, step = g.standard_normal(pre.shape), 1e-6
    diff = float(((B.gelu(pre + step * v) - B.gelu(pre - step * v)) * dy).sum() / (2 * step))
    assert abs(diff - float((dpre * v).sum())) <= 1e-7 * max(1.0, abs(diff))
    assert np.allclose(dbias, dpre.reshape(n, d, t).sum((0, 2)))
    x, w, u = g.standard_normal((n, c * t)), g.standard_normal((d, c, t)), g.standard_normal((d, c, t))
    diff = float(((oracle.fwd(x, w + step * u) - oracle.fwd(x, w - step * u)) * dy).sum() / (2 * step))
    assert abs(diff - float((B.bwd_w(x, dy, t) * u).sum())) <= 1e-6 * max(1.0, abs(diff))


def test_checkpoint_format():
    g = rng(9)
    x = g.standard_normal((7, 75)) * np.exp(4 * g.standard_normal((7, 1)))
    codes, scale = B.pack(x)
    assert codes.shape == (7, 96) and scale.shape == (7, 3)
    assert not codes[:, 75:].any()
    step = np.ldexp(1.0, scale.astype(int) - 127)
    back = B.unpack(codes, scale, 75)
    assert (np.abs(back - x) <= 0.5 * np.repeat(step, 32, axis=1)[:, :75]).all()
    # The step is the smallest that fits: the largest code takes seven bits.
    assert (np.abs(codes.reshape(7, 3, 32)).max(2) >= 64).all()
    # Packing what was unpacked changes nothing.
    codes2, scale2 = B.pack(back)
    assert np.array_equal(B.unpack(codes2, scale2, 75), back)


def test_checkpoint_boundaries():
    top = 127.5
    x = np.zeros((8, 32))
    x[0, 0] = np.nextafter(top, 0)   # just fits the unit step
    x[1, 0] = top                    # takes the next step
    x[2, 0], x[2, 1] = 64.0, 2.5     # unit step, a tie to the even code
    x[3, 0], x[3, 1] = 64.0, -3.5
    x[4, 5] = np.inf
    x[5, 6] = np.nan
    x[6, 0] = 2.0 ** -140            # far below the smallest step
    codes, scale = B.pack(x)
    assert list(scale[:, 0]) == [127, 128, 127, 127, 255, 255, 1, 1]
    assert codes[0, 0] == 127 and codes[1, 0] == 64 and codes[2, 1] == 2 and codes[3, 1] == -4
    assert not codes[6].any() and not codes[7].any()
    assert np.isnan(B.unpack(codes, scale, 32)[4:6]).all()
