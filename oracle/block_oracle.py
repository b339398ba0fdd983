"""fp64 NumPy definitions of the block operators (include/eqlinear_block.h): the equivariant layer
norm with its gradients, the 8-bit checkpoint format, and the gradients taken through it.
Used only by the tests; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np
from scipy.special import erf

BLOCK = 32


def norm(x, gamma, beta, T, eps):
    """(y, h, mean, rstd) of rows x [N, C*T]; gamma, beta [C] or None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = 1.0 / np.sqrt((centred ** 2).mean(1) + eps)
    h = centred * rstd[:, None]
    return affine(h, gamma, beta, T), h, mean, rstd


def affine(h, gamma, beta, T):
    g = 1.0 if gamma is None else np.repeat(np.asarray(gamma, np.float64), T)[None]
    b = 0.0 if beta is None else np.repeat(np.asarray(beta, np.float64), T)[None]
    return h * g + b


def norm_bwd(dy, h, rstd, gamma, T, dres=None):
    """(dx, dgamma, dbeta) for a given h and rstd."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    g = affine(dy, gamma, None, T)
    dx = np.asarray(rstd, np.float64)[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    per_channel = lambda v: v.reshape(v.shape[0], -1, T).sum((0, 2))  # noqa: E731
    return dx, per_channel(dy * h), per_channel(dy)


LAST_STEP = {"f32": 121, "f16": 9}  # exponent of the largest step of which 127 are finite


def pack(x, dtype="f32"):
    """(codes [N, P] int8, scale bytes [N, P / 32] uint8) of x [N, R] in `dtype`; the codes of a block
    with an infinity or a NaN are given as zeros (the format leaves them open)."""
    x = np.asarray(x, np.float64)
    n, r = x.shape
    p = -(-r // BLOCK) * BLOCK
    v = np.zeros((n, p))
    v[:, :r] = x
    v = v.reshape(n, p // BLOCK, BLOCK)
    finite = np.isfinite(v).all(2)
    v = np.where(finite[..., None], v, 0.0)
    top = np.abs(v).max(2)
    e = np.full(top.shape, -126)
    # The smallest e >= -126 with top < 127.5 * 2^e, found by counting up from below.
    e = np.where(top > 0, np.maximum(e, np.frexp(top)[1] - 9), e)
    for _ in range(4):
        e = np.where(top < np.ldexp(127.5, e), e, e + 1)
    held = e > LAST_STEP[dtype]
    e = np.minimum(e, LAST_STEP[dtype])
    codes = np.rint(np.ldexp(v, -e[..., None]))
    assert np.abs(codes[~held]).max(initial=0) <= 127
    codes = np.clip(codes, -127, 127)
    scale = np.where(finite, e + 127, 255).astype(np.uint8)
    return codes.astype(np.int8).reshape(n, p), scale


def buffer(codes, scale):
    """The checkpoint's bytes."""
    return np.concatenate([codes.view(np.uint8).reshape(-1), scale.reshape(-1)])


def unpack(codes, scale, r):
    step = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    n, p = codes.shape
    return (codes.reshape(n, -1, BLOCK) * step[..., None]).reshape(n, p)[:, :r]


def gelu(v):
    return 0.5 * v * (1.0 + erf(v / np.sqrt(2.0)))


def gelu_grad(v):
    return 0.5 * (1.0 + erf(v / np.sqrt(2.0))) + v * np.exp(-0.5 * v * v) / np.sqrt(2.0 * np.pi)


def gelu_bwd(dy, v, T):
    """(dpre, dbias) for GELU's input v."""
    dpre = np.asarray(dy, np.float64) * gelu_grad(v)
    return dpre, dpre.reshape(dpre.shape[0], -1, T).sum((0, 2))


def bwd_w(v, dy, T):
    """dw[d, c, t] = sum over n and g of dy[n, d, g] v[n, c, (g - t) mod T]."""
    v, dy = np.asarray(v, np.float64), np.asarray(dy, np.float64)
    dense = (dy.T @ v).reshape(dy.shape[1] // T, T, v.shape[1] // T, T)  # the unrolled layer's
    out = np.empty((dense.shape[0], dense.shape[2], T))
    for t in range(T):
        out[:, :, t] = sum(dense[:, g, :, (g - t) % T] for g in range(T))
    return out


def mlp_block(x, gamma, beta, w1, b1, w2, b2, eps, dy, ckpt8):
    """(y, gradients by name) of x + W2 gelu(W1 norm(x) + b1) + b2 for output gradient dy; ckpt8: the
    backward reads the normalised rows and GELU's input rounded to 8-bit checkpoints."""
    import oracle
    T = w1.shape[2]
    u, h, _, rstd = norm(x, gamma, beta, T, eps)
    pre = oracle.fwd(u, w1) + np.repeat(np.asarray(b1, np.float64), T)[None]
    y = np.asarray(x, np.float64) + oracle.fwd(gelu(pre), w2) + np.repeat(np.asarray(b2, np.float64), T)[None]
    if ckpt8:
        h, pre = (unpack(*pack(v), v.shape[1]) for v in (h, pre))
        u = affine(h, gamma, beta, T)
    dy = np.asarray(dy, np.float64)
    dpre, db1 = gelu_bwd(oracle.bwd_x(dy, w2), pre, T)
    dx, dgamma, dbeta = norm_bwd(oracle.bwd_x(dpre, w1), h, rstd, gamma, T, dy)
    return y, {"x": dx, "gamma": dgamma, "beta": dbeta, "w1": bwd_w(u, dpre, T), "b1": db1,
               "w2": bwd_w(gelu(pre), dy, T), "b2": dy.reshape(dy.shape[0], -1, T).sum((0, 2))}
