"""GPU parity of the layer in 8-bit integers (include/eqlinear_q8.h) against its fp64 definition
(oracle/q8_oracle.py).

Bounds, derived from the formulas.
  * Rows: a plane is a sum of T products in fp32, so within (T + 2) 2^-24 of the sum of magnitudes (the
    norm's weight another rounding); times 127 / m (two roundings) and to an integer: a code is within
    half of the fp64 plane's times 127 / m, plus that error times 127 / m, plus 127 * 2^-22.  At T = 1, 2 and 4 on fp16
    values the planes of these tests are exact and codes equal the oracle's.
  * The product is compared with the codes and scales that were written, read back: sums are exact;
    the sum's conversion, two scales and the inverse transform's T terms (twiddles within 2^-25) are
    within (T + 6) 2^-24 of the sum of the planes' magnitudes; bias and residual a rounding each; GELU within 2e-6.
    Results are rounded once: fp16 2^-11 of the value.
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
ULP = {"f16": 2.0 ** -11, "f32": 2.0 ** -24}
ACT = {"none": eql.EQL_ACT_NONE, "gelu": eql.EQL_ACT_GELU}
EPS = 1e-6

# (N, C, T): each lane arrangement and its last chunk, every group order, rows past the registers.
ROWS = [(1, 1, 1), (3, 15, 1), (70, 16, 1), (5, 1000, 1), (9, 4097, 1), (2, 20001, 1), (33, 9, 2), (7, 2050, 2), (1, 9000, 2),
        (65, 21, 3), (4, 1025, 3), (197, 96, 4), (1, 1024, 4), (6, 1025, 4), (2, 5000, 4), (31, 133, 5), (3, 2600, 5),
        (21, 40, 6), (17, 31, 7), (130, 64, 8), (5, 600, 8), (12, 66, 9), (3, 300, 10), (2, 1200, 11), (13, 71, 12),
        (4, 33, 13), (3, 260, 14), (11, 30, 15), (9, 65, 16), (2, 1100, 16)]
# (N, C, D, T): tails of every axis, one row, tall and wide, every group order.
PRODUCTS = [(1, 1, 1, 1), (1, 64, 32, 1), (5, 65, 33, 1), (33, 200, 100, 1), (1, 1024, 1024, 4), (2, 130, 70, 4), (197, 96, 384, 4),
            (40, 31, 17, 2), (3, 500, 40, 3), (64, 133, 171, 5), (65, 20, 50, 6), (31, 70, 40, 7), (129, 64, 64, 8),
            (7, 33, 66, 9), (40, 129, 20, 10), (17, 65, 35, 11), (66, 30, 31, 12), (5, 40, 33, 13), (33, 66, 9, 14),
            (9, 17, 65, 15), (35, 64, 32, 16), (1, 4000, 3, 4), (700, 3, 2, 4),
            (20, 1100, 70, 1), (70, 4130, 40, 1), (33, 1024, 64, 1),  # long sums in turns of four steps
            (1, 4200, 70, 1), (3, 1500, 40, 1)]  # few rows, long sums
# Enough tiles for the large kernel, ragged in every axis.
LARGE = [(1500, 70, 1050, 1), (1000, 130, 2100, 2), (1100, 65, 1700, 3), (1030, 100, 1999, 4), (2060, 64, 513, 5),
         (1030, 33, 1100, 6), (530, 130, 2048, 7), (700, 129, 1500, 8), (300, 65, 1700, 9), (300, 40, 1700, 10),
         (290, 64, 1700, 12), (513, 20, 1000, 15), (260, 66, 2100, 16), (16500, 96, 96, 4), (4100, 20, 40, 8),
         # Both tiles of the large kernel, and odd and even numbers of K blocks.
         (4200, 450, 1810, 1), (2060, 470, 2020, 2), (500, 70, 1000, 3), (500, 200, 1000, 4), (1100, 290, 1700, 4)]


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def scratch(nbytes):
    return torch.full((max(int(nbytes), 16),), 0xFF, dtype=torch.uint8, device=DEV)


def rows_of(x, n, c, t, dtype):
    buf = scratch(eql.eqlinear_q8_rows_bytes(n, c, t))
    eql.eqlinear_q8_quantize(x, buf, n, c, t, DT[dtype])
    return buf


def weight_of(w, d, c, t, dtype):
    buf = scratch(eql.eqlinear_q8_weight_bytes(d, c, t))
    eql.eqlinear_q8_pack_weight(w, buf, d, c, t, DT[dtype])
    return buf


def read_weight(buf, D, C, T):
    """(codes [T, D, C], scales [D, F] without the inverse transform's share) of a packed weight; its
    padding is checked to be zero.  Codes: [block of 32 outputs][block of 64 inputs][T][2][half][output][16]."""
    buf = buf.cpu().numpy()
    ob, kb, F = -(-D // 32), -(-C // 64), T // 2 + 1
    n = ob * kb * T * 2048
    codes = buf[:n].view(np.int8).reshape(ob, kb, T, 2, 2, 32, 16)
    codes = codes.transpose(2, 0, 5, 1, 3, 4, 6).reshape(T, ob * 32, kb * 64)
    assert not codes[:, D:].any() and not codes[:, :, C:].any()
    scales = buf[n:n + F * ob * 128].view(np.float32).reshape(F, ob * 32)
    assert not scales[:, D:].any()
    real = 2 if T % 2 == 0 and T > 1 else 1
    share = np.where(np.arange(F) < real, 1.0, 2.0)[:, None] / T
    return codes[:, :D, :C], (scales[:, :D] / share).T.astype(np.float64)


def check_codes(codes, scales, pl, mags, T, exact, rstd_off=0.0):
    """Codes and scales against planes [T, rows, C] with the sums' magnitudes `mags` [rows, C]."""
    rc, rs = Q.encode(pl, T)
    for f, where in enumerate(Q.frequencies(T)[1]):
        if exact:
            assert np.array_equal(codes[where], rc[where])
            assert (np.abs(scales[:, f] - rs[:, f]) <= 2.0 ** -23 * rs[:, f]).all()
            continue
        m = np.maximum(np.abs(pl[where]).max((0, 2)), Q.FLOOR)
        err = (T + 4) * 2.0 ** -24 * mags.max(1)
        assert (np.abs(scales[:, f] * 127.0 - m) <= err + (2.0 ** -22 + rstd_off) * m).all()
        want = pl[where] * (127.0 / m)[:, None]
        slack = 0.5 + 127.0 * (2.0 ** -22 + (2 * err / m)[:, None])
        assert (np.abs(codes[where].astype(np.float64) - want) <= slack).all()
        assert np.abs(codes[where].astype(int)).max() <= 127


def values(n, c, t, dtype, seed):
    g = np.random.default_rng([seed, n, c, t])
    # Multiples of 2^-6 below 16: exact in fp16, and any sums of them in fp32.
    v = np.round(g.standard_normal((n, c, t)) * 2.0 ** 6) * 2.0 ** -6 + 0.25
    return v.astype(NP[dtype])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_quantize(shape, dtype):
    n, c, t = shape
    print("case q8 rows", shape, dtype, flush=True)
    x = values(n, c, t, dtype, 0)
    codes, scales, pad = Q.read_rows(rows_of(dev(x.reshape(n, -1)), n, c, t, dtype).cpu().numpy(), n, c, t)
    assert not pad.any()
    check_codes(codes, scales, Q.planes(x, t), np.abs(x.astype(np.float64)).sum(2), t, t in (1, 2, 4))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_norm_rows(shape, residual, dtype):
    n, c, t = shape
    print("case q8 norm", shape, residual, dtype, flush=True)
    x, r = values(n, c, t, dtype, 1), values(n, c, t, dtype, 2)
    gamma = (1 + 0.2 * np.random.default_rng(5).standard_normal(c)).astype(NP[dtype])
    kept = (x.astype(np.float64) + r.astype(np.float64)).astype(NP[dtype]) if residual else x
    buf, s = scratch(eql.eqlinear_q8_rows_bytes(n, c, t)), torch.empty(n, c * t, dtype=dev(x).dtype, device=DEV)
    xd, rd = dev(x.reshape(n, -1)), dev(r.reshape(n, -1)) if residual else None
    eql.eqlinear_q8_rmsnorm(xd, rd, dev(gamma), s, buf, n, c, t, EPS, DT[dtype])
    assert np.array_equal(s.cpu().numpy(), kept.reshape(n, -1))
    codes, scales, pad = Q.read_rows(buf.cpu().numpy(), n, c, t)
    assert not pad.any()
    rstd = Q.rmsnorm(kept.reshape(n, -1), None, t, EPS)[2]
    k64, g64 = kept.astype(np.float64), gamma.astype(np.float64)
    mags = np.abs(k64).sum(2) * np.abs(g64)
    scales = scales / rstd[:, None]
    if t not in (1, 2, 4):
        # The scales hold rstd, which is within 1e-5 (the row's sum).
        check_codes(codes, scales, Q.planes(k64, t) * g64[None, None], mags, t, False, 1e-5)
    else:
        # The planes are exact in fp32, times the weight rounded once.
        rc, rs = Q.encode((Q.planes(k64, t).astype(np.float32) * gamma.astype(np.float32)[None, None]).astype(np.float64), t)
        assert np.array_equal(codes, rc)
        assert (np.abs(scales - rs) <= 1e-5 * rs).all()
    # Without the sum, in place, and without a weight.
    for kw in ("none", "x", "res"):
        if kw == "res" and not residual:
            continue
        a, b, again = xd.clone(), rd.clone() if residual else None, scratch(buf.numel())
        target = {"none": None, "x": a, "res": b}[kw]
        eql.eqlinear_q8_rmsnorm(a, b, dev(gamma), target, again, n, c, t, EPS, DT[dtype])
        assert torch.equal(again, buf)
        if target is not None:
            assert torch.equal(target, s)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (40, 70, 1), (33, 65, 2), (5, 130, 3), (100, 64, 4), (7, 9, 5), (31, 200, 8),
                                   (64, 33, 12), (3, 66, 16)], ids=str)
def test_pack_weight(shape, dtype):
    d, c, t = shape
    w = values(d, c, t, dtype, 3)
    codes, scales = read_weight(weight_of(dev(w), d, c, t, dtype), d, c, t)
    check_codes(codes, scales, Q.planes(w, t), np.abs(w.astype(np.float64)).sum(2), t, t in (1, 2, 4))


def product_case(n, c, d, t, dtype, seed):
    g = np.random.default_rng([seed, n, c, d, t])
    x = (g.standard_normal((n, c * t)) * np.exp(0.3 * g.standard_normal((1, c * t)))).astype(NP[dtype])
    w = (g.standard_normal((d, c, t)) / np.sqrt(c * t)).astype(NP[dtype])
    return x, w, (0.3 * g.standard_normal(d)).astype(NP[dtype]), g.standard_normal((n, d * t)).astype(NP[dtype])


def check_product(rows8, w8, y, bias, act, res, n, c, d, t, dtype):
    xc, xs, _ = Q.read_rows(rows8.cpu().numpy(), n, c, t)
    wc, ws = read_weight(w8, d, c, t)
    # Sums of whole numbers below 2^53: exact, so that one that cancels is zero here too.
    xp, wp = xc.astype(np.float64), wc.astype(np.float64)
    pl, mags = np.zeros((t, n, d)), np.zeros((n, d))
    for f, where in enumerate(Q.frequencies(t)[1]):
        unit = np.outer(xs[:, f], ws[:, f])
        if len(where) == 1:
            pl[where[0]] = xp[where[0]] @ wp[where[0]].T * unit
            mags += np.abs(pl[where[0]]) / t
        else:
            (xr, xi), (wr, wi) = xp[where], wp[where]
            pl[where[0]], pl[where[1]] = (xr @ wr.T - xi @ wi.T) * unit, (xr @ wi.T + xi @ wr.T) * unit
            mags += 2.0 / t * (np.abs(pl[where[0]]) + np.abs(pl[where[1]]))
    lay = Q.values(pl, t)
    ref = Q.epilogue(lay, bias, act, res)
    slack = (t + 6) * 2.0 ** -24 * mags[..., None] + 2.0 ** -23 * np.abs(lay)
    slack = np.broadcast_to(slack, lay.shape).reshape(n, -1) * 1.13  # GELU's slope is at most 1.13
    slack = slack + 2.0 ** -23 * (np.abs(ref) + (0.0 if res is None else np.abs(res)) + (0.0 if bias is None else np.repeat(np.abs(bias), t)))
    if act == "gelu":
        slack = slack + 2e-6
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    bound = ULP[dtype] * np.abs(ref) + slack + (2.0 ** -25 if dtype == "f16" else 1e-37)
    assert (err <= bound).all(), "off by up to %.3g times the bound" % (err / bound).max()


def run_product(rows8, w8, bias, act, res, n, c, d, t, dtype):
    y = torch.empty(n, d * t, dtype=torch.float16 if dtype == "f16" else torch.float32, device=DEV)
    eql.eqlinear_q8_fwd(rows8, w8, bias, res, y, n, c, d, t, DT[dtype], ACT[act])
    return y


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", PRODUCTS + LARGE, ids=str)
def test_product(shape, dtype):
    n, c, d, t = shape
    print("case q8 product", shape, dtype, flush=True)
    x, w, b, r = product_case(n, c, d, t, dtype, 0)
    rows8, w8 = rows_of(dev(x), n, c, t, dtype), weight_of(dev(w), d, c, t, dtype)
    for bias, act, res in ((None, "none", None), (b, "gelu", None), (b, "none", r), (None, "gelu", r)):
        y = run_product(rows8, w8, dev(bias), act, dev(res), n, c, d, t, dtype)
        check_product(rows8, w8, y, bias, act, res, n, c, d, t, dtype)
    y2 = dev(r)  # the residual's place
    eql.eqlinear_q8_fwd(rows8, w8, None, y2, y2, n, c, d, t, DT[dtype], ACT["gelu"])
    assert torch.equal(y, y2)


@pytest.mark.parametrize("shape", [(700, 96, 384, 4), (1500, 70, 1050, 1), (600, 64, 700, 8), (260, 40, 900, 12), (1100, 65, 1700, 3)], ids=str)
def test_rows_do_not_depend_on_each_other(shape):
    """A row's outputs are the same bits alone, among a few and among many: sums are exact."""
    n, c, d, t = shape
    x, w, b, r = product_case(n, c, d, t, "f16", 1)
    w8 = weight_of(dev(w), d, c, t, "f16")
    whole = run_product(rows_of(dev(x), n, c, t, "f16"), w8, dev(b), "gelu", dev(r), n, c, d, t, "f16")
    for lo, hi in ((0, 1), (n - 1, n), (7, 10), (3, 40), (5, 205)):
        part = run_product(rows_of(dev(x[lo:hi]), hi - lo, c, t, "f16"), w8, dev(b), "gelu", dev(r[lo:hi]), hi - lo, c, d, t, "f16")
        assert torch.equal(part, whole[lo:hi])


@pytest.mark.parametrize("t", [1, 2, 4])
def test_group_shift(t):
    """A cyclic shift of the input's group axis shifts the output, bit for bit."""
    n, c, d = 50, 40, 36
    x = values(n, c, t, "f16", 6)
    w = values(d, c, t, "f16", 7)
    w8 = weight_of(dev(w), d, c, t, "f16")
    y, ys = (run_product(rows_of(dev(v.reshape(n, -1)), n, c, t, "f16"), w8, None, "none", None, n, c, d, t, "f16")
             for v in (x, np.roll(x, 1, axis=2)))
    assert np.array_equal(np.roll(y.cpu().numpy().reshape(n, d, t), 1, axis=2), ys.cpu().numpy().reshape(n, d, t))


@pytest.mark.parametrize("t", [1, 3, 4, 8])
def test_accuracy_of_the_whole(t):
    """Against the unrounded layer.  Each factor's error is at most half a scale, uniformly spread: a
    scale is m / 127 with m below six times the plane's root mean square here, so 6 / 127 / sqrt(12) =
    1.4% of it each, 1.9% for both, 2.5% with the tails' allowance."""
    n, c, d = 300, 256, 80
    g = np.random.default_rng(t)
    x, w = g.standard_normal((n, c, t)).astype(np.float16), (g.standard_normal((d, c, t)) / 16).astype(np.float16)
    y = run_product(rows_of(dev(x.reshape(n, -1)), n, c, t, "f16"), weight_of(dev(w), d, c, t, "f16"), None, "none", None, n, c, d, t, "f16")
    ref = Q.layer(x.astype(np.float64), w.astype(np.float64)).reshape(n, -1)
    err = np.linalg.norm(y.cpu().numpy().astype(np.float64) - ref) / np.linalg.norm(ref)
    assert 1e-3 < err < 0.025


@pytest.mark.parametrize("n", [9, 2000])
@pytest.mark.parametrize("t", [1, 4, 5])
def test_special_values(t, n):
    """Zero rows give the bias; an infinity or a NaN takes its row, or its output channel, and no other;
    values below the scales' floor count as zero."""
    c, d = 40, 600
    x, w, b, _ = product_case(n, c, d, t, "f32", 3)
    x[1], x[2, 3], x[3, 5 % (c * t)], x[4] = 0.0, np.inf, np.nan, x[4] * 2.0 ** -140
    w[7, 2, 0], w[8, 1, 0], w[9] = np.nan, -np.inf, 0.0
    rows8, w8 = rows_of(dev(x), n, c, t, "f32"), weight_of(dev(w), d, c, t, "f32")
    y = run_product(rows8, w8, dev(b), "none", None, n, c, d, t, "f32").cpu().numpy().reshape(n, d, t)
    assert np.isnan(y[2:4]).all() and np.isnan(y[:, 7:9]).all()
    y[:, 7:9], y[2:4] = 0.0, 0.0
    assert np.isfinite(y).all()
    plain = np.broadcast_to(b[:, None], (d, t)).copy()
    plain[7:9] = 0.0
    assert np.array_equal(y[1], plain) and np.array_equal(y[4], plain)
    assert np.array_equal(y[5, 9], np.full(t, b[9]))


def test_large_values():
    """fp32 rows near the type's end: planes that stay finite give finite outputs, one that overflows NaN."""
    c, d, t = 20, 9, 4
    x = np.ones((3, c, t), np.float32)
    x[0] *= 2.0 ** 125   # the sum of four is 2^127
    x[1] *= 2.0 ** 126   # 2^128 is infinite
    w = np.full((d, c, t), 2.0 ** -20, np.float32)
    y = run_product(rows_of(dev(x.reshape(3, -1)), 3, c, t, "f32"), weight_of(dev(w), d, c, t, "f32"), None, "none", None, 3, c, d, t, "f32")
    got = y.cpu().numpy()
    assert np.allclose(got[0], 2.0 ** 125 * 2.0 ** -20 * c * t, rtol=1e-5) and np.isnan(got[1]).all()
    assert np.allclose(got[2], 2.0 ** -20 * c * t, rtol=1e-5)


def test_largest_sums():
    """Codes of 127 throughout at the channel limit: the complex planes' sums come to 2 C 127^2, below 2^31."""
    c, d, t, n = 65536, 2, 4, 2
    x = np.zeros((n, c, t), np.float16)
    x[..., 0], x[..., 1] = 1.0, -1.0     # X1 = 1 + i: re = im = 127
    w = np.zeros((d, c, t), np.float16)
    w[..., 0], w[..., 1] = 2.0 ** -6, 2.0 ** -6  # W1 = (1 - i) / 64: re = 127, im = -127
    rows8, w8 = rows_of(dev(x.reshape(n, -1)), n, c, t, "f16"), weight_of(dev(w), d, c, t, "f16")
    codes, _, _ = Q.read_rows(rows8.cpu().numpy(), n, c, t)
    assert (codes[2] == 127).all() and (codes[3] == 127).all()
    y = run_product(rows8, w8, None, "none", None, n, c, d, t, "f16")
    ref = Q.layer(x[:1].astype(np.float64), w[:1].astype(np.float64)).reshape(-1)  # (x0 w0, ...) c times
    assert np.array_equal(y.cpu().numpy().astype(np.float64).reshape(n * d, t), np.broadcast_to(ref, (n * d, t)))


def test_streams_and_graph():
    """The whole chain on another stream, and captured and replayed with eager work between."""
    n, c, d, t = 197, 96, 384, 4
    x, w, b, _ = product_case(n, c, d, t, "f16", 4)
    r, gamma = dev(product_case(n, c, d, t, "f16", 5)[0]), dev(np.ones(c, np.float16))
    xd, bd, w8 = dev(x), dev(b), weight_of(dev(w), d, c, t, "f16")
    s, rows8 = torch.empty_like(xd), scratch(eql.eqlinear_q8_rows_bytes(n, c, t))
    y = torch.empty(n, d * t, dtype=torch.float16, device=DEV)

    def run(s, rows8, y):
        eql.eqlinear_q8_rmsnorm(xd, r, gamma, s, rows8, n, c, t, EPS, DT["f16"])
        eql.eqlinear_q8_fwd(rows8, w8, bd, None, y, n, c, d, t, DT["f16"], ACT["gelu"])
    run(s, rows8, y)
    want = [v.clone() for v in (s, rows8, y)]
    side = torch.cuda.Stream()
    for v in (s, rows8, y):
        v.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(s, rows8, y)
    torch.cuda.current_stream().wait_stream(side)
    for got, ref in zip((s, rows8, y), want):
        assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(s, rows8, y)
    fresh = [torch.empty_like(v) for v in (s, rows8, y)]
    for k in range(4):
        xd.copy_(dev(product_case(n, c, d, t, "f16", 10 + k)[0]))
        graph.replay()
        torch.cuda.synchronize()
        run(*fresh)
        for got, ref in zip((s, rows8, y), fresh):
            assert torch.equal(got, ref)


def test_guards():
    """Nothing is written past a buffer's end: canaries behind every output stay."""
    for n, c, d, t in ((3, 33, 35, 4), (5, 20, 7, 3), (200, 16, 40, 1), (1050, 40, 600, 5)):
        x, w, b, r = product_case(n, c, d, t, "f16", 6)
        nr, nw, ny = eql.eqlinear_q8_rows_bytes(n, c, t), eql.eqlinear_q8_weight_bytes(d, c, t), n * d * t * 2
        rows8, w8, y = (torch.full((k + 512,), 0x5A, dtype=torch.uint8, device=DEV) for k in (nr, nw, ny))
        eql.eqlinear_q8_quantize(dev(x), rows8, n, c, t, DT["f16"])
        eql.eqlinear_q8_pack_weight(dev(w), w8, d, c, t, DT["f16"])
        eql.eqlinear_q8_fwd(rows8, w8, dev(b), dev(r), y, n, c, d, t, DT["f16"], ACT["none"])
        for buf, k in ((rows8, nr), (w8, nw), (y, ny)):
            assert (buf[k:] == 0x5A).all()
