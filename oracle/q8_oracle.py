"""fp64 NumPy definitions of the RMS norm (include/eqlinear_rmsnorm.h) and of the layer in 8-bit
integers (include/eqlinear_q8.h).  Used only by the tests; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np
from scipy.special import erf

FLOOR = 2.0 ** -100


def rmsnorm(s, gamma, T, eps):
    """(y, h, rstd) of rows s [N, C*T] (the sum as it is kept); gamma [C] or None."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    h = s * rstd[:, None]
    return h * spread(gamma, T), h, rstd


def spread(gamma, T):
    return 1.0 if gamma is None else np.repeat(np.asarray(gamma, np.float64), T)[None]


def rmsnorm_bwd(dy, h, rstd, gamma, T, dres=None):
    """(dx, dgamma)."""
    dy = np.asarray(dy, np.float64)
    g = dy * spread(gamma, T)
    dx = rstd[:, None] * (g - h * (g * h).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * h).reshape(dy.shape[0], -1, T).sum((0, 2))


def frequencies(T):
    """The frequencies in the order of the scales, and each one's planes."""
    ks = [0] + ([T // 2] if T > 1 and T % 2 == 0 else [])
    real = len(ks)
    where = [[i] for i in range(real)] + [[real + 2 * q, real + 2 * q + 1] for q in range((T - real) // 2)]
    return ks + list(range(1, (T - real) // 2 + 1)), where


def planes(v, T):
    """[rows, C, T] -> [T, rows, C] real planes of the half spectrum."""
    v = np.asarray(v, np.float64)
    out = np.zeros((T,) + v.shape[:2])
    t = np.arange(T)
    for k, where in zip(*frequencies(T)):
        angle = 2.0 * np.pi * ((k * t) % T) / T
        out[where[0]] = v @ np.cos(angle)
        if len(where) == 2:
            out[where[1]] = -(v @ np.sin(angle))
    return out


def values(pl, T):
    """Planes [T, rows, C] -> [rows, C, T]."""
    out = np.zeros(pl.shape[1:] + (T,))
    t = np.arange(T)
    for k, where in zip(*frequencies(T)):
        angle = 2.0 * np.pi * ((k * t) % T) / T
        if len(where) == 1:
            out += pl[where[0]][..., None] * np.cos(angle) / T
        else:
            out += 2.0 * (pl[where[0]][..., None] * np.cos(angle) - pl[where[1]][..., None] * np.sin(angle)) / T
    return out


def encode(pl, T):
    """Codes [T, rows, C] and scales [rows, F] of planes, the codes' operations (1 / m, 127 times it, the plane times
    that), each in fp32."""
    _, groups = frequencies(T)
    codes, scales = np.zeros(pl.shape, np.int8), np.zeros((pl.shape[1], len(groups)))
    for f, where in enumerate(groups):
        p = pl[where].astype(np.float32)
        m = np.maximum(np.abs(p).max((0, 2)), np.float32(FLOOR))
        inv = np.float32(127.0) * (np.float32(1.0) / m)
        codes[where] = np.rint(p * inv[:, None])
        scales[:, f] = m.astype(np.float64) / 127.0
    return codes, scales


def decode(codes, scales, T):
    """The planes that codes [T, rows, C] and scales [rows, F] stand for."""
    out = codes.astype(np.float64)
    for f, where in enumerate(frequencies(T)[1]):
        out[where] *= scales[:, f][:, None]
    return out


def read_rows(buf, N, C, T):
    """(codes [T, N, C], scales [N, F], padding [N, T, P - C]) of a buffer of 8-bit rows."""
    P, F = -(-C // 16) * 16, T // 2 + 1
    buf = np.ascontiguousarray(buf)
    codes = buf[:N * T * P].view(np.int8).reshape(N, T, P)
    scales = buf[N * T * P:N * T * P + N * F * 4].view(np.float32).reshape(N, F)
    return codes[..., :C].transpose(1, 0, 2), scales.astype(np.float64), codes[..., C:]


def layer(x, w):
    """y [N, D, T] of x [N, C, T] and w [D, C, T]: y[n, d, g] = sum w[d, c, (g - h) mod T] x[n, c, h]."""
    T = x.shape[2]
    y = np.zeros((x.shape[0], w.shape[0], T))
    for g in range(T):
        for h in range(T):
            y[:, :, g] += x[:, :, h] @ w[:, :, (g - h) % T].T
    return y


def epilogue(y, bias, act, residual):
    """act(y + bias) + residual on [N, D, T], as rows."""
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[:, None]
    if act == "gelu":
        y = 0.5 * y * (1.0 + erf(y / np.sqrt(2.0)))
    y = y.reshape(y.shape[0], -1)
    return y if residual is None else y + np.asarray(residual, np.float64)
