"""GPU parity of the block operators (include/eqlinear_block.h) against their fp64 definitions
(oracle/block_oracle.py): the equivariant layer norm, forward and backward, 8-bit checkpoints,
and the passes that read them.

Bounds, derived from the formulas:
  * fp16 results are rounded once, 2^-11 of the value (2^-25 below the normal range);
  * fp32 arithmetic: a row's sums run over chains of at most 64 additions and ten joins, a
    column's over at most 128 additions and 32 joins in these tests, each within 2^-24, so
    errors stay below 1e-5 of the sum of magnitudes;
  * a rational approximation of erf within 1.5e-7, so GELU and its slope within 2e-6;
  * weight gradients: the layer's own bounds, 1e-5 (fp32) and 3e-3 (fp16) of the norm.
"""
import numpy as np
import pytest
import torch

import group_circulant_linear_p4_amd as eql
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NP = {"f16": np.float16, "f32": np.float32}
DT = {"f16": eql.EQL_F16, "f32": eql.EQL_F32}
ULP = {"f16": 2.0 ** -11, "f32": 0.0}
EPS = 1e-5
F32ERR = 1e-5

# (N, C, T): one feature; short rows; every lane arrangement and its last chunk; rows that no
# 8 or 32 divides; rows past what the registers hold, backward (8192) and forward (16384).
SHAPES = [(1, 1, 1), (1, 5, 3), (3, 8, 4), (197, 96, 4), (33, 171, 3), (64, 133, 5), (17, 64, 8), (2500, 16, 1),
          (1100, 3, 16), (300, 7, 1), (129, 129, 4), (70, 512, 4), (41, 513, 4), (9, 1024, 4), (6, 1500, 4), (5, 2048, 4),
          (3, 2731, 3), (700, 8200, 1), (2, 4099, 4), (1, 20011, 1), (12, 96, 4), (50, 99, 2), (21, 66, 9), (13, 400, 12),
          (4, 700, 12), (11, 300, 15), (515, 31, 7)]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.cpu().numpy().astype(np.float64)


def scratch(nbytes):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=DEV)


def close(got, ref, slack, dtype):
    """|got - ref| <= one rounding of ref + slack, element by element; NaN where ref is."""
    got = host(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    err = np.abs(got - ref)
    bound = ULP[dtype] * np.abs(ref) + slack + (2.0 ** -25 if dtype == "f16" else 1e-37)
    ok = (err <= bound) | np.isnan(ref)
    assert ok.all(), "off by up to %.3g times the bound" % np.nanmax(err / bound)


def activations(g, n, r, dtype):
    x = g.standard_normal((n, r)) * np.exp(0.5 * g.standard_normal((1, r))) + 0.3 * g.standard_normal((n, 1))
    x[g.random(n) < 0.05] *= 16
    return x.astype(NP[dtype])


def run_norm(x, gamma, beta, dtype, c, t, ckpt=True, stats=True, inplace=False, stream=None):
    n = x.shape[0]
    y = x if inplace else torch.empty_like(x)
    ck = scratch(eql.eqlinear_ckpt8_bytes(n, c, t)) if ckpt else None
    mean = torch.empty(n, dtype=torch.float32, device=DEV) if stats else None
    rstd = torch.empty(n, dtype=torch.float32, device=DEV) if stats else None
    eql.eqlinear_layernorm_fwd(x, gamma, beta, y, ck, mean, rstd, n, c, t, EPS, DT[dtype], stream)
    return y, ck, mean, rstd


def ckpt_parts(ck, n, r):
    p = -(-r // 32) * 32
    raw = ck.cpu().numpy()
    return raw[:n * p].view(np.int8).reshape(n, p), raw[n * p:n * (p + p // 32)].reshape(n, p // 32)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm_forward(shape, dtype):
    n, c, t = shape
    print("case norm forward", shape, dtype, flush=True)
    g = np.random.default_rng(n * 7 + c)
    x = activations(g, n, c * t, dtype)
    gamma, beta = (1 + 0.2 * g.standard_normal(c)).astype(NP[dtype]), (0.1 * g.standard_normal(c)).astype(NP[dtype])
    y, ck, mean, rstd = run_norm(dev(x), dev(gamma), dev(beta), dtype, c, t)
    ry, rh, rmean, rrstd = B.norm(x, gamma, beta, t, EPS)
    wide = np.abs(x.astype(np.float64)).max(1)
    # The mean is off by rounding of the largest features, times rstd in h.
    herr = F32ERR * (np.abs(rh).max(1) + rrstd * wide)
    assert (np.abs(host(mean) - rmean) <= F32ERR * wide).all()
    assert (np.abs(host(rstd) - rrstd) <= 2 * F32ERR * rrstd * (1 + rrstd * wide)).all()
    gl = np.abs(gamma.astype(np.float64)).max()
    close(y, ry, (2 * herr * gl + F32ERR * np.abs(ry).max(1))[:, None], dtype)
    # The checkpoint of h: every value within half its block's step, steps as small as the
    # largest magnitude allows, nothing past the row's end.
    codes, scale = ckpt_parts(ck, n, c * t)
    assert not codes[:, c * t:].any() and (codes != -128).all()
    step = np.repeat(np.ldexp(1.0, scale.astype(int) - 127), 32, axis=1)[:, :c * t]
    assert (np.abs(B.unpack(codes, scale, c * t) - rh) <= 0.5 * step + herr[:, None]).all()
    top = np.abs(codes.astype(int)).reshape(n, -1, 32).max(2)
    assert ((top >= 63) | (scale == 1)).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_norm_optional_arguments_and_in_place(dtype):
    n, c, t = 37, 50, 4
    g = np.random.default_rng(3)
    x = activations(g, n, c * t, dtype)
    gamma, beta = g.standard_normal(c).astype(NP[dtype]), g.standard_normal(c).astype(NP[dtype])
    for ga, be in ((gamma, None), (None, beta), (None, None)):
        y, _, _, _ = run_norm(dev(x), None if ga is None else dev(ga), None if be is None else dev(be), dtype, c, t,
                              ckpt=False, stats=False)
        ry, rh, _, rr = B.norm(x, ga, be, t, EPS)
        close(y, ry, 1e-4 * np.abs(ry).max(), dtype)
    full = run_norm(dev(x), dev(gamma), dev(beta), dtype, c, t)[0]
    assert torch.equal(run_norm(dev(x), dev(gamma), dev(beta), dtype, c, t, inplace=True)[0], full)
    for n2, c2 in ((3, 20011),):  # the path of long rows
        x2 = activations(g, n2, c2, dtype)
        assert torch.equal(run_norm(dev(x2), None, None, dtype, c2, 1)[0], run_norm(dev(x2), None, None, dtype, c2, 1, inplace=True)[0])


def run_norm_bwd(dy, src, mean, rstd, gamma, dres, dtype, c, t, params=True, dx=None, stream=None):
    n = dy.shape[0]
    dx = torch.empty_like(dy) if dx is None else dx
    dg = torch.empty(c, dtype=dy.dtype, device=DEV) if params else None
    db = torch.empty(c, dtype=dy.dtype, device=DEV) if params else None
    nbytes = eql.eqlinear_layernorm_bwd_workspace_bytes(n, c, t, DT[dtype])
    ws = scratch(nbytes)
    if mean is None:
        eql.eqlinear_layernorm_bwd_ckpt8(dy, src, rstd, gamma, dres, dx, dg, db, ws, nbytes, n, c, t, DT[dtype], stream)
    else:
        eql.eqlinear_layernorm_bwd(dy, src, mean, rstd, gamma, dres, dx, dg, db, ws, nbytes, n, c, t, DT[dtype], stream)
    return dx, dg, db


def check_norm_bwd(got, dy, h, herr, rstd, gamma, dres, c, t, dtype):
    dx, dg, db = got
    rdx, rdg, rdb = B.norm_bwd(dy, h, rstd, gamma, t, dres)
    gd = np.abs(B.affine(np.asarray(dy, np.float64), gamma, None, t))
    ha = np.abs(h)
    r = dy.shape[1]
    size = gd.max(1) + ha.max(1) * (gd * ha).sum(1) / r
    # h itself is off by herr: in m2, and times m2.
    slack = rstd * (3 * F32ERR * size + herr * 2 * (gd.max(1) + (gd * ha).sum(1) / r)) + F32ERR * np.abs(rdx).max(1)
    close(dx, rdx, slack[:, None], dtype)
    per = lambda v: v.reshape(v.shape[0], -1, t).sum((0, 2))  # noqa: E731
    ad = np.abs(np.asarray(dy, np.float64))
    close(dg, rdg, F32ERR * per(ad * ha) + per(ad * herr[:, None]) + 1e-30, dtype)
    close(db, rdb, F32ERR * per(ad) + 1e-30, dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("source", ["x", "ckpt"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm_backward(shape, source, dtype):
    n, c, t = shape
    print("case norm backward", shape, source, dtype, flush=True)
    g = np.random.default_rng(n * 11 + c)
    r = c * t
    x = activations(g, n, r, dtype)
    gamma = (1 + 0.2 * g.standard_normal(c)).astype(NP[dtype])
    dy, dres = (0.05 * g.standard_normal((n, r))).astype(NP[dtype]), (0.05 * g.standard_normal((n, r))).astype(NP[dtype])
    _, h, mean, rstd = B.norm(x, gamma, None, t, EPS)
    rs = rstd.astype(np.float32)
    if source == "ckpt":
        codes, scale = B.pack(h)
        h, herr = B.unpack(codes, scale, r), np.zeros(n)
        got = run_norm_bwd(dev(dy), dev(B.buffer(codes, scale)), None, dev(rs), dev(gamma), dev(dres), dtype, c, t)
    else:
        mn = mean.astype(np.float32)
        herr = 2.0 ** -22 * (np.abs(x.astype(np.float64)).max(1) * rstd + np.abs(h).max(1))
        got = run_norm_bwd(dev(dy), dev(x), dev(mn), dev(rs), dev(gamma), dev(dres), dtype, c, t)
    check_norm_bwd(got, dy, h, herr, rs.astype(np.float64), gamma, dres, c, t, dtype)


@pytest.mark.parametrize("shape", [(37, 50, 4), (5, 1024, 4), (3, 8200, 1)], ids=str)
def test_norm_backward_optional_arguments_and_in_place(shape):
    n, c, t = shape
    g = np.random.default_rng(5)
    r = c * t
    x = activations(g, n, r, "f16")
    dy, dres = g.standard_normal((n, r)).astype(np.float16), g.standard_normal((n, r)).astype(np.float16)
    gamma = g.standard_normal(c).astype(np.float16)
    y, ck, mean, rstd = run_norm(dev(x), dev(gamma), None, "f16", c, t)
    for src, mn in ((dev(x), mean), (ck, None)):
        full = run_norm_bwd(dev(dy), src, mn, rstd, dev(gamma), dev(dres), "f16", c, t)
        alone = run_norm_bwd(dev(dy), src, mn, rstd, dev(gamma), dev(dres), "f16", c, t, params=False)
        assert torch.equal(alone[0], full[0])
        d = dev(dy)
        over = run_norm_bwd(d, src, mn, rstd, dev(gamma), dev(dres), "f16", c, t, dx=d)
        assert all(torch.equal(a, b) for a, b in zip(over, full))
        e = dev(dres)
        over = run_norm_bwd(dev(dy), src, mn, rstd, dev(gamma), e, "f16", c, t, dx=e)
        assert all(torch.equal(a, b) for a, b in zip(over, full))
        bare = run_norm_bwd(dev(dy), src, mn, rstd, None, None, "f16", c, t)
        ones = run_norm_bwd(dev(dy), src, mn, rstd, dev(np.ones(c, np.float16)), dev(np.zeros((n, r), np.float16)), "f16", c, t)
        assert all(torch.equal(a, b) for a, b in zip(bare, ones))


def test_no_rows():
    empty = torch.empty((0, 20), dtype=torch.float16, device=DEV)
    dg, db = (torch.full((5,), 7.0, dtype=torch.float16, device=DEV) for _ in range(2))
    one = torch.empty(1, dtype=torch.float32, device=DEV)
    eql.eqlinear_layernorm_fwd(empty, None, None, empty, None, None, None, 0, 5, 4, EPS, eql.EQL_F16)
    eql.eqlinear_layernorm_bwd(empty, empty, one, one, None, None, empty, dg, db, None, 0, 0, 5, 4, eql.EQL_F16)
    assert not dg.any().item() and not db.any().item()
    dg.fill_(7.0)
    eql.eqlinear_layernorm_bwd_ckpt8(empty, None, one, None, None, empty, dg, None, None, 0, 0, 5, 4, eql.EQL_F16)
    assert not dg.any().item()
    db.fill_(7.0)
    eql.eqlinear_fused_epilogue_bwd_ckpt8(empty, None, empty, db, None, 0, 0, 5, 4, eql.EQL_F16)
    assert not db.any().item()
    dw = torch.full((3, 5, 4), 7.0, dtype=torch.float16, device=DEV)
    eql.eqlinear_bwd_w_ckpt8(None, None, None, eql.EQL_ACT_NONE, None, dw, None, 0, 0, 5, 3, 4, eql.EQL_F16)
    assert not dw.any().item()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_checkpoint_pack_and_unpack(shape, dtype):
    """Codes and scale bytes equal the definition's bit for bit; the values come back exactly."""
    n, c, t = shape
    r = c * t
    g = np.random.default_rng(n + c)
    x = (g.standard_normal((n, r)) * np.exp2(g.integers(-8, 8, (n, 1)))).astype(NP[dtype])
    x[:, ::7] = np.round(x[:, ::7] * 4) / 4   # ties
    if r > 40:
        x[0, :32] = 0
        x[-1, 33] = 127.5
    ck = scratch(eql.eqlinear_ckpt8_bytes(n, c, t))
    ck.fill_(77)
    eql.eqlinear_ckpt8_pack(dev(x), ck, n, c, t, DT[dtype])
    codes, scale = B.pack(x)
    got_codes, got_scale = ckpt_parts(ck, n, r)
    assert np.array_equal(got_scale, scale) and np.array_equal(got_codes, codes)
    back = torch.empty((n, r), dtype=torch.float16 if dtype == "f16" else torch.float32, device=DEV)
    eql.eqlinear_ckpt8_unpack(ck, back, n, c, t, DT[dtype])
    assert np.array_equal(back.cpu().numpy(), B.unpack(codes, scale, r).astype(NP[dtype]))


def test_checkpoint_special_values():
    """Non-finite blocks read back as NaN and their neighbours do not; the extremes of fp32."""
    x = np.zeros((9, 100), np.float32)
    x[:, :] = 0.25
    x[0, 5], x[1, 40], x[2, 99] = np.inf, np.nan, -np.inf
    x[3, :32] = np.finfo(np.float32).max
    x[4, :32] = -np.finfo(np.float32).tiny
    x[5, :32] = 1e-45
    x[6, 3] = 127.5
    x[7, 3] = np.nextafter(np.float32(127.5), np.float32(0))
    x[8, :32] = 0
    x[8, 3] = -0.0
    ck = scratch(eql.eqlinear_ckpt8_bytes(9, 100, 1))
    eql.eqlinear_ckpt8_pack(dev(x), ck, 9, 100, 1, eql.EQL_F32)
    codes, scale = B.pack(x)
    got_codes, got_scale = ckpt_parts(ck, 9, 100)
    assert np.array_equal(got_scale, scale)
    fine = np.repeat(scale != 255, 32, axis=1)
    assert np.array_equal(got_codes[fine], codes[fine])
    back = torch.empty((9, 100), dtype=torch.float32, device=DEV)
    eql.eqlinear_ckpt8_unpack(ck, back, 9, 100, 1, eql.EQL_F32)
    assert np.array_equal(back.cpu().numpy(), B.unpack(codes, scale, 100).astype(np.float32), equal_nan=True)


def test_non_finite_rows_stay_in_their_rows():
    n, c, t = 12, 40, 4
    g = np.random.default_rng(8)
    x = activations(g, n, c * t, "f16")
    x[2, 7], x[5, 0], x[9, 159] = np.nan, np.inf, -np.inf
    dy = g.standard_normal((n, c * t)).astype(np.float16)
    y, ck, mean, rstd = run_norm(dev(x), None, None, "f16", c, t)
    bad = np.zeros(n, bool)
    bad[[2, 5, 9]] = True
    assert np.array_equal(np.isnan(host(y)).all(1), bad) and np.array_equal(np.isnan(host(y)).any(1), bad)
    codes, scale = ckpt_parts(ck, n, c * t)
    assert (scale[bad] == 255).all() and (scale[~bad] != 255).all()
    for src, mn in ((dev(x), mean), (ck, None)):
        dx, dg, db = run_norm_bwd(dev(dy), src, mn, rstd, None, None, "f16", c, t)
        assert np.array_equal(np.isnan(host(dx)).all(1), bad) and np.array_equal(np.isnan(host(dx)).any(1), bad)
        assert torch.isnan(dg).all().item() and torch.isfinite(db).all().item()


@pytest.mark.parametrize("shape", [(3, 4, 1), (5, 8, 1), (9, 24, 4), (6, 13, 1), (2, 8193, 1), (2, 10000, 1)], ids=str)
def test_constant_rows_of_large_values(shape):
    """h is zero, though mean rstd is beyond fp32: y = beta, dx = rstd (g - mean(g))."""
    n, c, t = shape
    r, eps, f32 = c * t, 1e-12, eql.EQL_F32
    g = np.random.default_rng(c)
    dy = g.standard_normal((n, r)).astype(np.float32)
    gamma, beta = (g.standard_normal(c).astype(np.float32) for _ in range(2))
    x, y = torch.full((n, r), 2.0 ** 110, dtype=torch.float32, device=DEV), torch.empty((n, r), device=DEV)
    mean, rstd = (torch.empty(n, dtype=torch.float32, device=DEV) for _ in range(2))
    eql.eqlinear_layernorm_fwd(x, dev(gamma), dev(beta), y, None, mean, rstd, n, c, t, eps, f32)
    assert np.array_equal(y.cpu().numpy(), np.broadcast_to(np.repeat(beta, t), (n, r)))
    dx, dg, db = run_norm_bwd(dev(dy), x, mean, rstd, dev(gamma), None, "f32", c, t)
    rdx, _, rdb = B.norm_bwd(dy, np.zeros((n, r)), np.full(n, 1e6), gamma, t, None)
    close(dx, rdx, F32ERR * 1e6 * np.abs(dy * np.repeat(gamma, t)).max(), "f32")
    assert not dg.any().item()
    close(db, rdb, F32ERR * np.abs(dy).sum(), "f32")


GELU_SHAPES = [(1, 1, 1), (3, 8, 4), (197, 384, 4), (501, 171, 3), (64, 133, 5), (2500, 16, 1), (30, 700, 3), (9, 2051, 4),
               (3001, 40, 4), (700, 300, 7), (20, 900, 16),
               (64, 700, 4), (65, 700, 4), (33, 640, 5), (17, 100, 16), (64, 2100, 1),
               # column blocks of whole channels at orders that do not divide 8
               (100, 900, 7), (300, 601, 15), (40, 1200, 9), (35, 1367, 12), (600, 2733, 3), (1, 5461, 3), (50, 1, 13)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", GELU_SHAPES, ids=str)
def test_gelu_backward(shape, dtype):
    n, d, t = shape
    print("case gelu backward", shape, dtype, flush=True)
    g = np.random.default_rng(n + d)
    codes, scale = B.pack(1.5 * g.standard_normal((n, d * t)))
    v = B.unpack(codes, scale, d * t)
    dy = g.standard_normal((n, d * t)).astype(NP[dtype])
    nbytes = eql.eqlinear_fused_epilogue_bwd_workspace_bytes(n, d, t, DT[dtype])
    dy_d, ck = dev(dy), dev(B.buffer(codes, scale))
    dpre, db, ws = torch.empty_like(dy_d), torch.empty(d, dtype=dy_d.dtype, device=DEV), scratch(nbytes)
    eql.eqlinear_fused_epilogue_bwd_ckpt8(dy_d, ck, dpre, db, ws, nbytes, n, d, t, DT[dtype])
    rdpre, rdb = B.gelu_bwd(dy, v, t)
    ady = np.abs(dy.astype(np.float64))
    close(dpre, rdpre, 2e-6 * ady, dtype)
    close(db, rdb, (2e-6 + 1.2 * F32ERR) * ady.reshape(n, d, t).sum((0, 2)), dtype)
    alone = torch.empty_like(dy_d)
    eql.eqlinear_fused_epilogue_bwd_ckpt8(dy_d, ck, alone, None, None, 0, n, d, t, DT[dtype])
    assert torch.equal(alone, dpre)
    eql.eqlinear_fused_epilogue_bwd_ckpt8(dy_d, ck, dy_d, db, ws, nbytes, n, d, t, DT[dtype])
    assert torch.equal(dy_d, dpre)


# Both weight-gradient paths, every group order's code alignment, ragged channels, one row.
WEIGHT = [(197, 96, 40, 4), (1, 3, 5, 4), (700, 70, 90, 4), (100, 21, 17, 1), (64, 40, 8, 2), (90, 11, 13, 3),
          (33, 7, 9, 5), (50, 6, 12, 6), (40, 5, 5, 7), (129, 64, 64, 8), (21, 5, 3, 9), (17, 4, 4, 10), (19, 3, 5, 11),
          (70, 8, 6, 12), (23, 3, 3, 13), (15, 5, 4, 14), (31, 2, 6, 15), (44, 6, 10, 16), (300, 1024, 1024, 4)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", WEIGHT, ids=str)
def test_weight_gradient(shape, dtype):
    n, c, d, t = shape
    print("case weight gradient", shape, dtype, flush=True)
    g = np.random.default_rng(n + c + d)
    codes, scale = B.pack(g.standard_normal((n, c * t)))
    value = B.unpack(codes, scale, c * t)
    dy = g.standard_normal((n, d * t)).astype(NP[dtype])
    gamma, beta = (1 + 0.2 * g.standard_normal(c)).astype(NP[dtype]), (0.1 * g.standard_normal(c)).astype(NP[dtype])
    nbytes = eql.eqlinear_bwd_w_workspace_bytes(n, c, d, t, DT[dtype])
    dy_d, ck, ws = dev(dy), dev(B.buffer(codes, scale)), scratch(nbytes)
    for ga, be, act in ((None, None, "none"), (gamma, beta, "none"), (None, None, "gelu"), (gamma, None, "gelu")):
        v = B.affine(value, ga, be, t)
        v = B.gelu(v) if act == "gelu" else v
        dw = torch.empty((d, c, t), dtype=dy_d.dtype, device=DEV)
        eql.eqlinear_bwd_w_ckpt8(ck, None if ga is None else dev(ga), None if be is None else dev(be),
                                 eql.EQL_ACT_GELU if act == "gelu" else eql.EQL_ACT_NONE, dy_d, dw, ws, nbytes, n, c, d, t,
                                 DT[dtype])
        ref = B.bwd_w(v, dy, t)
        rel = np.linalg.norm(host(dw) - ref) / np.linalg.norm(ref)
        assert rel <= (1e-5 if dtype == "f32" else 3e-3), (act, rel)


@pytest.mark.parametrize("shape,dtype", [((4096, 96, 40, 4), "f16"), ((1500, 512, 512, 4), "f16"), ((500, 24, 40, 8), "f32")], ids=str)
def test_spectrum_in_a_training_step(shape, dtype):
    """The checkpoint's spectrum beside the input gradient's: the same weight gradient."""
    n, c, d, t = shape
    g = np.random.default_rng(c)
    codes, scale = B.pack(g.standard_normal((n, c * t)))
    v = B.gelu(B.unpack(codes, scale, c * t))
    dy = g.standard_normal((n, d * t)).astype(NP[dtype])
    w = (g.standard_normal((d, c, t)) / np.sqrt(c * t)).astype(NP[dtype])
    code = DT[dtype]
    nbytes = eql.eqlinear_bwd_w_workspace_bytes(n, c, d, t, code)
    ws, dy_d = scratch(nbytes), dev(dy)
    wp = scratch(eql.eqlinear_packed_weight_bytes(c, d, t, code))
    eql.eqlinear_pack_weight(dev(w), wp, d, c, t, code, eql.EQL_PACK_BWDX)
    dx = torch.empty((n, c * t), dtype=dy_d.dtype, device=DEV)
    dw = torch.empty((d, c, t), dtype=dy_d.dtype, device=DEV)
    eql.eqlinear_ckpt8_spectrum(dev(B.buffer(codes, scale)), None, None, eql.EQL_ACT_GELU, ws, nbytes, n, c, d, t, code)
    eql.eqlinear_bwd_x_train(dy_d, wp, dx, ws, nbytes, n, c, d, t, code)
    eql.eqlinear_bwd_w_train(dy_d, dw, ws, nbytes, n, c, d, t, code)
    ref = B.bwd_w(v, dy, t)
    assert np.linalg.norm(host(dw) - ref) / np.linalg.norm(ref) <= (1e-5 if dtype == "f32" else 3e-3)


def test_results_repeat_on_another_stream_and_in_a_graph():
    """Every operator twice, on a stream of its own, and replayed from a graph between eager
    work: bit-identical."""
    n, c, t = 1031, 48, 4
    g = np.random.default_rng(2)
    x, gamma = dev(activations(g, n, c * t, "f16")), dev(np.ones(c, np.float16))
    dy = dev(g.standard_normal((n, c * t)).astype(np.float16))
    dw = torch.empty((c, c, t), dtype=torch.float16, device=DEV)
    y, dx, dpre = (torch.empty_like(x) for _ in range(3))
    dg, db, dbias = (torch.empty(c, dtype=torch.float16, device=DEV) for _ in range(3))
    ck, ck2 = (scratch(eql.eqlinear_ckpt8_bytes(n, c, t)) for _ in range(2))
    rstd = torch.empty(n, dtype=torch.float32, device=DEV)
    sizes = (eql.eqlinear_layernorm_bwd_workspace_bytes(n, c, t, eql.EQL_F16),
             eql.eqlinear_fused_epilogue_bwd_workspace_bytes(n, c, t, eql.EQL_F16),
             eql.eqlinear_bwd_w_workspace_bytes(n, c, c, t, eql.EQL_F16))
    ws = [scratch(b) for b in sizes]
    outs = (y, dx, dpre, dg, db, dbias, dw, ck, ck2, rstd)

    def step():
        eql.eqlinear_layernorm_fwd(x, gamma, None, y, ck, None, rstd, n, c, t, EPS, eql.EQL_F16)
        eql.eqlinear_ckpt8_pack(y, ck2, n, c, t, eql.EQL_F16)
        eql.eqlinear_layernorm_bwd_ckpt8(dy, ck, rstd, gamma, dy, dx, dg, db, ws[0], sizes[0], n, c, t, eql.EQL_F16)
        eql.eqlinear_fused_epilogue_bwd_ckpt8(dx, ck2, dpre, dbias, ws[1], sizes[1], n, c, t, eql.EQL_F16)
        eql.eqlinear_bwd_w_ckpt8(ck, gamma, None, eql.EQL_ACT_GELU, dpre, dw, ws[2], sizes[2], n, c, c, t, eql.EQL_F16)

    def wipe():
        for o in outs:
            o.view(torch.uint8).fill_(85)

    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    wipe()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        wipe()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_past_32_bits():
    """More than 2^31 features in all: the last rows equal those of the same rows alone."""
    c, t, tail = 1024, 4, 3
    n = (1 << 31) // (c * t) + 4099
    print("case offsets past 32 bits: %d rows of %d" % (n, c * t), flush=True)
    torch.manual_seed(1)
    x = torch.empty((n, c * t), dtype=torch.float16, device=DEV)
    x[:] = torch.randn(1, c * t, device=DEV).half()
    x[-tail:] = torch.randn(tail, c * t, device=DEV).half()
    last = x[-tail:].clone()
    y, ck, mean, rstd = run_norm(x, None, None, "f16", c, t)
    y1, ck1, mean1, rstd1 = run_norm(last, None, None, "f16", c, t)
    assert torch.equal(y[-tail:], y1) and torch.equal(rstd[-tail:], rstd1) and torch.equal(mean[-tail:], mean1)
    p, b = c * t, c * t // 32
    assert torch.equal(ck[(n - tail) * p:n * p], ck1[:tail * p])
    assert torch.equal(ck[n * p + (n - tail) * b:], ck1[tail * p:])
    back, back1 = torch.empty_like(x), torch.empty_like(last)
    eql.eqlinear_ckpt8_unpack(ck, back, n, c, t, eql.EQL_F16)
    eql.eqlinear_ckpt8_unpack(ck1, back1, tail, c, t, eql.EQL_F16)
    assert torch.equal(back[-tail:], back1)
    ck2 = scratch(eql.eqlinear_ckpt8_bytes(n, c, t))
    eql.eqlinear_ckpt8_pack(back, ck2, n, c, t, eql.EQL_F16)
    assert torch.equal(ck2, ck)
    for src, mn, src1, mn1 in ((x, mean, last, mean1), (ck, None, ck1, None)):
        dx, _, _ = run_norm_bwd(y, src, mn, rstd, None, back, "f16", c, t, dx=back if mn is None else None)
        dx1, _, _ = run_norm_bwd(y1, src1, mn1, rstd1, None, back1, "f16", c, t)
        assert torch.equal(dx[-tail:], dx1)
    nbytes = eql.eqlinear_fused_epilogue_bwd_workspace_bytes(n, c, t, eql.EQL_F16)
    ws, db = scratch(nbytes), torch.empty(c, dtype=torch.float16, device=DEV)
    eql.eqlinear_fused_epilogue_bwd_ckpt8(y, ck, back, db, ws, nbytes, n, c, t, eql.EQL_F16)
    eql.eqlinear_fused_epilogue_bwd_ckpt8(y1, ck1, back1, None, None, 0, tail, c, t, eql.EQL_F16)
    assert torch.equal(back[-tail:], back1)
