"""GPU parity of the RMS norm (include/eqlinear_rmsnorm.h) against its fp64 definition
(oracle/q8_oracle.py).

Bounds, derived from the formulas: fp16 results are rounded once, 2^-11 of the value (2^-25 below the
normal range).  fp32 arithmetic: a row's sum runs over chains of at most 128 additions and ten joins,
a column's over at most 128 additions and 32 joins in these tests, each within 2^-24, so errors stay
below 1e-5 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import group_circulant_linear_p4_amd as eql
from oracle import q8_oracle as Q

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NP = {"f16": np.float16, "f32": np.float32}
DT = {"f16": eql.EQL_F16, "f32": eql.EQL_F32}
ULP = {"f16": 2.0 ** -11, "f32": 0.0}
EPS = 1e-6
F32ERR = 1e-5

# (N, C, T): one feature; short rows; every lane arrangement and its last chunk; rows that no 8
# divides; rows past what the registers hold, backward (8192) and forward (16384).
SHAPES = [(1, 1, 1), (1, 5, 3), (3, 8, 4), (197, 96, 4), (33, 171, 3), (64, 133, 5), (17, 64, 8), (2500, 16, 1),
          (1100, 3, 16), (300, 7, 1), (129, 129, 4), (70, 512, 4), (41, 513, 4), (9, 1024, 4), (1, 1024, 4), (6, 1500, 4),
          (5, 2048, 4), (3, 2731, 3), (700, 8200, 1), (2, 4099, 4), (1, 20011, 1), (50, 99, 2), (13, 400, 12), (11, 300, 15),
          (515, 31, 7)]


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.cpu().numpy().astype(np.float64)


def scratch(nbytes):
    return torch.full((max(int(nbytes), 16),), 0xFF, dtype=torch.uint8, device=DEV)


def close(got, ref, slack, dtype):
    """|got - ref| <= one rounding of ref + slack, element by element; NaN where ref is."""
    got = host(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bound = ULP[dtype] * np.abs(ref) + slack + (2.0 ** -25 if dtype == "f16" else 1e-37)
    err = np.abs(got - ref)
    assert ((err <= bound) | np.isnan(ref)).all(), "off by up to %.3g times the bound" % np.nanmax(err / bound)


def case(n, c, t, dtype, seed=0):
    g = np.random.default_rng([seed, n, c, t])
    r = c * t
    x = (g.standard_normal((n, r)) * np.exp(0.5 * g.standard_normal((1, r))) + 0.3).astype(NP[dtype])
    res, dy, dres = (g.standard_normal((n, r)).astype(NP[dtype]) for _ in range(3))
    return x, res, (1 + 0.2 * g.standard_normal(c)).astype(NP[dtype]), dy, dres


def forward(x, res, gamma, n, c, t, dtype, sum=True, rstd=True):
    s = torch.empty_like(x) if sum else None
    y, rs = torch.empty_like(x), torch.empty(n, device=DEV) if rstd else None
    eql.eqlinear_rmsnorm_fwd(x, res, gamma, s, y, rs, n, c, t, EPS, DT[dtype])
    return s, y, rs


def backward(dy, s, rstd, gamma, dres, n, c, t, dtype, params=True):
    dx = torch.empty_like(dy)
    dg = torch.empty(c, dtype=dy.dtype, device=DEV) if params else None
    nb = eql.eqlinear_rmsnorm_bwd_workspace_bytes(n, c, t, DT[dtype])
    eql.eqlinear_rmsnorm_bwd(dy, s, rstd, gamma, dres, dx, dg, scratch(nb), nb, n, c, t, DT[dtype])
    return dx, dg


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, dtype):
    n, c, t = shape
    print("case rmsnorm", shape, dtype, flush=True)
    x, res, gamma, dy, dres = case(n, c, t, dtype)
    s, y, rstd = forward(dev(x), dev(res), dev(gamma), n, c, t, dtype)
    kept = (x.astype(np.float64) + res.astype(np.float64)).astype(NP[dtype])
    assert np.array_equal(s.cpu().numpy(), kept)  # one addition, rounded once
    ry, h, rr = Q.rmsnorm(kept, gamma, t, EPS)
    close(y, ry, F32ERR * np.abs(ry), dtype)
    close(rstd, rr, F32ERR * rr, "f32")
    dx, dg = backward(dev(dy), s, rstd, dev(gamma), dev(dres), n, c, t, dtype)
    rdx, rdg = Q.rmsnorm_bwd(dy, h, rr, gamma, t, dres)
    g = np.abs(dy.astype(np.float64)) * np.repeat(np.abs(gamma.astype(np.float64)), t)
    close(dx, rdx, F32ERR * (rr[:, None] * (g + np.abs(h) * (g * np.abs(h)).mean(1, keepdims=True)) + np.abs(dres)), dtype)
    close(dg, rdg, F32ERR * (np.abs(dy) * np.abs(h)).reshape(n, c, t).sum((0, 2)), dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", [(5, 12, 4), (197, 96, 4), (3, 2731, 3), (2, 20011, 1)], ids=str)
def test_optional_operands(shape, dtype):
    """Without a residual, a weight, the sum or rstd: what is left computes the same."""
    n, c, t = shape
    x, res, gamma, dy, dres = case(n, c, t, dtype, 1)
    kept = (x.astype(np.float64) + res.astype(np.float64)).astype(NP[dtype])
    s, y, rstd = forward(dev(x), dev(res), dev(gamma), n, c, t, dtype)
    _, y2, _ = forward(dev(x), dev(res), dev(gamma), n, c, t, dtype, sum=False, rstd=False)
    assert torch.equal(y, y2)
    s3, y3, _ = forward(dev(kept), None, dev(gamma), n, c, t, dtype)
    assert torch.equal(y, y3) and torch.equal(s3, s)
    _, y4, _ = forward(dev(kept), None, None, n, c, t, dtype)
    _, y5, _ = forward(dev(kept), None, dev(np.ones_like(gamma)), n, c, t, dtype)
    assert torch.equal(y4, y5)
    full = backward(dev(dy), s, rstd, dev(gamma), dev(dres), n, c, t, dtype)
    assert torch.equal(full[0], backward(dev(dy), s, rstd, dev(gamma), dev(dres), n, c, t, dtype, params=False)[0])
    none = backward(dev(dy), s, rstd, dev(gamma), None, n, c, t, dtype)
    zero = backward(dev(dy), s, rstd, dev(gamma), dev(np.zeros_like(dres)), n, c, t, dtype)
    assert torch.equal(none[0], zero[0]) and torch.equal(none[1], zero[1])


@pytest.mark.parametrize("shape", [(5, 12, 4), (197, 96, 4), (41, 133, 5), (3, 2731, 3), (2, 20011, 1)], ids=str)
def test_in_place(shape):
    """sum, y and dx written over their inputs."""
    n, c, t = shape
    x, res, gamma, dy, dres = case(n, c, t, "f16", 2)
    s, y, rstd = forward(dev(x), dev(res), dev(gamma), n, c, t, "f16")
    for over in ("x", "res"):
        a, b, yo = dev(x), dev(res), torch.empty_like(y)
        target = a if over == "x" else b
        eql.eqlinear_rmsnorm_fwd(a, b, dev(gamma), target, yo, None, n, c, t, EPS, DT["f16"])
        assert torch.equal(target, s) and torch.equal(yo, y)
        a, b, so = dev(x), dev(res), torch.empty_like(y)
        target = a if over == "x" else b
        eql.eqlinear_rmsnorm_fwd(a, b, dev(gamma), so, target, None, n, c, t, EPS, DT["f16"])
        assert torch.equal(target, y) and torch.equal(so, s)
    dx, dg = backward(dev(dy), s, rstd, dev(gamma), dev(dres), n, c, t, "f16")
    nb = eql.eqlinear_rmsnorm_bwd_workspace_bytes(n, c, t, DT["f16"])
    for over in ("dy", "dres"):
        a, b = dev(dy), dev(dres)
        target = a if over == "dy" else b
        eql.eqlinear_rmsnorm_bwd(a, s, rstd, dev(gamma), b, target, None, scratch(nb), nb, n, c, t, DT["f16"])
        assert torch.equal(target, dx)


def test_special_rows():
    """Zero rows, infinities, NaN and squares past fp32, each among ordinary rows."""
    n, c, t = 9, 24, 4
    x, res, gamma, dy, _ = case(n, c, t, "f32", 3)
    res[1], x[1] = 0.0, 0.0
    x[2, 5], x[3, 7], x[4, 0] = np.inf, np.nan, 1e30
    x[5] *= 1e-20
    res[5] = 0.0
    s, y, rstd = forward(dev(x), dev(res), dev(gamma), n, c, t, "f32")
    ry, _, _ = Q.rmsnorm((x + res).astype(np.float32), gamma, t, EPS)
    got = host(y)
    assert not got[1].any() and np.isnan(got[2:5]).all()
    ok = [0, 1, 5, 6, 7, 8]
    close(y[ok], ry[ok], F32ERR * np.abs(ry[ok]), "f32")
    # Without eps a row of zeros has no direction.
    z = torch.zeros(2, c * t, device=DEV)
    out = torch.empty_like(z)
    eql.eqlinear_rmsnorm_fwd(z, None, dev(gamma), None, out, None, 2, c, t, 0.0, DT["f32"])
    assert torch.isnan(out).all()


def test_group_shift():
    """A cyclic shift of every channel's group axis shifts the result, bit for bit up to the row's sum."""
    n, c, t = 30, 20, 4
    x, res, gamma, _, _ = case(n, c, t, "f16", 4)
    roll = lambda a: np.roll(a.reshape(n, c, t), 1, axis=2).reshape(n, c * t)  # noqa: E731
    _, y, _ = forward(dev(x), dev(res), dev(gamma), n, c, t, "f16")
    _, ys, _ = forward(dev(roll(x)), dev(roll(res)), dev(gamma), n, c, t, "f16")
    ref = roll(host(y))
    assert (np.abs(host(ys) - ref) <= 2.0 ** -10 * np.abs(ref)).all()  # one step of fp16


def test_streams_and_graph():
    """On another stream, and captured and replayed with eager work between."""
    n, c, t = 300, 96, 4
    x, res, gamma, dy, dres = (dev(a) for a in case(n, c, t, "f16", 5))
    s, y, rstd = forward(x, res, gamma, n, c, t, "f16")
    dx, dg = backward(dy, s, rstd, gamma, dres, n, c, t, "f16")
    side = torch.cuda.Stream()
    nb = eql.eqlinear_rmsnorm_bwd_workspace_bytes(n, c, t, DT["f16"])
    bufs = [torch.empty_like(a) for a in (s, y, rstd, dx, dg)] + [scratch(nb)]

    def run():
        eql.eqlinear_rmsnorm_fwd(x, res, gamma, bufs[0], bufs[1], bufs[2], n, c, t, EPS, DT["f16"])
        eql.eqlinear_rmsnorm_bwd(dy, bufs[0], bufs[2], gamma, dres, bufs[3], bufs[4], bufs[5], nb, n, c, t, DT["f16"])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    for got, ref in zip(bufs, (s, y, rstd, dx, dg)):
        assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        x.copy_(dev(case(n, c, t, "f16", 10 + k)[0]))
        graph.replay()
        torch.cuda.synchronize()
        es, ey, er = forward(x, res, gamma, n, c, t, "f16")
        edx, edg = backward(dy, es, er, gamma, dres, n, c, t, "f16")
        for got, ref in zip(bufs, (es, ey, er, edx, edg)):
            assert torch.equal(got, ref)


def test_no_rows():
    c, t = 6, 4
    dg = torch.full((c,), 7.0, device=DEV)
    e = torch.empty(0, c * t, device=DEV)
    eql.eqlinear_rmsnorm_fwd(e, None, None, None, e, None, 0, c, t, EPS, DT["f32"])
    eql.eqlinear_rmsnorm_bwd(e, e, None, None, None, e, dg, None, 0, 0, c, t, DT["f32"])
    assert not dg.any()
