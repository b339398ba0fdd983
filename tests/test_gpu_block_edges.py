"""GPU tests of the block operators' edges (include/eqlinear_block.h): what the definitions give
exactly, and results at the ends of the number ranges."""
import numpy as np
import pytest
import torch

import group_circulant_linear_p4_amd as eql
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NP = {"f16": np.float16, "f32": np.float32}
DT = {"f16": eql.EQL_F16, "f32": eql.EQL_F32}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def scratch(nbytes):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=DEV)


# Row lengths R whose rounded reciprocal is not their inverse, fl(R fl(1 / R)) != 1: on 16 and on 64
# lanes and on a whole workgroup, one to several chunks a lane, whole and ragged rows, group orders
# with and without a table, and rows past the registers, backward (8192) and forward (16384).
UNEVEN = [(41, 1), (41, 4), (55, 3), (94, 2), (82, 4), (332, 2), (23, 5), (141, 4), (2256, 1), (614, 4), (8437, 1),
          (4331, 2), (16707, 1), (5774, 3), (3502, 5)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", UNEVEN, ids=str)
def test_constant_rows_have_no_deviation(shape, dtype):
    """The sum of R equal features is exact here (integers below 2^24 times a power of two), so the
    mean is the feature itself: h = 0, y = beta bit for bit, the checkpoint's codes are zero."""
    c, t = shape
    r, n = c * t, 5
    assert np.float32(r) * np.float32(1.0 / r) != 1
    g = np.random.default_rng(r)
    beta, gamma = (g.standard_normal(c).astype(NP[dtype]) for _ in range(2))
    for value in (1000.0, 16384.0) if dtype == "f16" else (1000.0, 16384.0, 2.0 ** 110):
        x = torch.full((n, r), value, dtype=torch.float16 if dtype == "f16" else torch.float32, device=DEV)
        y, ck = torch.empty_like(x), scratch(eql.eqlinear_ckpt8_bytes(n, c, t))
        mean, rstd = (torch.empty(n, dtype=torch.float32, device=DEV) for _ in range(2))
        eql.eqlinear_layernorm_fwd(x, dev(gamma), dev(beta), y, ck, mean, rstd, n, c, t, 1e-5, DT[dtype])
        assert (mean == value).all().item()
        assert np.array_equal(y.cpu().numpy(), np.broadcast_to(np.repeat(beta, t), (n, r)))
        assert not ck[:n * (-(-r // 32) * 32)].any().item()


@pytest.mark.parametrize("source", ["x", "ckpt"])
@pytest.mark.parametrize("shape", UNEVEN, ids=str)
def test_constant_gradients_of_constant_rows_vanish(shape, source):
    """With h = 0 and equal g the input gradient rstd (g - mean(g)) is zero, and so is dgamma; dbeta
    is the count."""
    c, t = shape
    r, n, f32 = c * t, 3, eql.EQL_F32
    dy, dx = torch.ones((n, r), device=DEV), torch.full((n, r), 7.0, device=DEV)
    x, mean, rstd = torch.full((n, r), 1000.0, device=DEV), torch.full((n,), 1000.0, device=DEV), torch.full((n,), 300.0, device=DEV)
    dg, db = torch.full((c,), 7.0, device=DEV), torch.empty(c, device=DEV)
    nbytes = eql.eqlinear_layernorm_bwd_workspace_bytes(n, c, t, f32)
    ws = scratch(nbytes)
    if source == "x":
        eql.eqlinear_layernorm_bwd(dy, x, mean, rstd, None, None, dx, dg, db, ws, nbytes, n, c, t, f32)
    else:
        ck = dev(B.buffer(*B.pack(np.zeros((n, r)))))
        eql.eqlinear_layernorm_bwd_ckpt8(dy, ck, rstd, None, None, dx, dg, db, ws, nbytes, n, c, t, f32)
    assert not dx.any().item() and not dg.any().item() and (db == n * t).all().item()


@pytest.mark.parametrize("shape", [(41, 4), (16707, 1)], ids=str)
def test_rows_whose_sum_overflows_are_nan(shape):
    """The other rows are not touched by it."""
    c, t = shape
    n, r = 4, c * t
    x = torch.randn(n, r, device=DEV)
    x[2] = 3e38
    y = torch.empty_like(x)
    eql.eqlinear_layernorm_fwd(x, None, None, y, None, None, None, n, c, t, 1e-5, eql.EQL_F32)
    assert torch.isnan(y[2]).all().item() and torch.isfinite(y[[0, 1, 3]]).all().item()


# Largest magnitudes of a block around the last one whose step the element type can hold.
TOPS = {"f16": [65184.0, 65248.0, 65280.0, 65312.0, 65472.0, 65504.0],
        "f32": [float(np.float32(v)) for v in (127.25 * 2.0 ** 121, np.nextafter(np.float32(127.5 * 2.0 ** 121), np.float32(0)),
                                               127.5 * 2.0 ** 121, 127.9 * 2.0 ** 121, np.finfo(np.float32).max)]}


@pytest.mark.parametrize("shape", [(3, 25, 4), (2, 32, 1), (5, 7, 5)], ids=str)
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_checkpoints_of_the_largest_finite_values(dtype, shape):
    """Finite matrices come back finite, each value within 1 / 127 of its block's largest."""
    n, c, t = shape
    r = c * t
    g = np.random.default_rng(r)
    for top in TOPS[dtype]:
        x = (top * g.uniform(-1, 1, (n, r))).astype(NP[dtype])
        x[0, :] = -top
        x[-1, ::3] = top
        ck, back = scratch(eql.eqlinear_ckpt8_bytes(n, c, t)), dev(np.zeros_like(x))
        eql.eqlinear_ckpt8_pack(dev(x), ck, n, c, t, DT[dtype])
        eql.eqlinear_ckpt8_unpack(ck, back, n, c, t, DT[dtype])
        got, x64 = back.cpu().numpy().astype(np.float64), x.astype(np.float64)
        assert np.isfinite(got).all(), top
        pad = np.zeros((n, -(-r // 32) * 32))
        pad[:, :r] = np.abs(x64)
        largest = np.repeat(pad.reshape(n, -1, 32).max(2), 32, axis=1)[:, :r]
        assert (np.abs(got - x64) <= largest / 127).all(), top
        codes, scale = B.pack(x, dtype)
        raw, p = ck.cpu().numpy(), codes.shape[1]
        assert np.array_equal(raw[:n * p].view(np.int8).reshape(n, p), codes)
        assert np.array_equal(raw[n * p:n * (p + p // 32)].reshape(n, -1), scale)
        # The passes that read a checkpoint see finite values too.
        dy, dpre = dev(np.ones_like(x)), dev(np.zeros_like(x))
        eql.eqlinear_fused_epilogue_bwd_ckpt8(dy, ck, dpre, None, None, 0, n, c, t, DT[dtype])
        assert torch.isfinite(dpre).all().item()
        if t == 1:  # one feature a channel: the spectrum is the input itself
            d, nbytes = 3, eql.eqlinear_bwd_w_workspace_bytes(n, c, 3, t, DT[dtype])
            e = np.zeros((n, d), NP[dtype])
            e[0, 1] = e[1, 2] = 1
            dw = torch.empty((d, c, t), dtype=back.dtype, device=DEV)
            eql.eqlinear_bwd_w_ckpt8(ck, None, None, eql.EQL_ACT_NONE, dev(e), dw, scratch(nbytes), nbytes, n, c, d, t, DT[dtype])
            assert np.array_equal(dw.cpu().numpy()[1:, :, 0], back.cpu().numpy()[:2])




def plain_spectrum_f16(x, t):
    """[T planes][N][C] as the transform computes them: sums over h in order, multiply-adds in fp32
    with coefficients rounded to fp32, 0 and +-1 exact; the last multiply-add rounds to fp16 once, a
    last addition to fp32 and then to fp16."""
    n = x.shape[0]
    v = x.astype(np.float32).reshape(n, -1, t).astype(np.longdouble)
    cs = [np.longdouble(np.float32(np.cos(2 * np.pi * m / t))) for m in range(t)]
    sn = [np.longdouble(np.float32(np.sin(2 * np.pi * m / t))) for m in range(t)]
    real = 2 if t % 2 == 0 and t > 1 else 1
    planes = []
    for p in range(t):
        k = 0 if p == 0 else (t // 2 if p < real else (p - real) // 2 + 1)
        imag = p >= real and (p - real) & 1
        terms = []  # (coefficient, needs a product)
        for h in range(t):
            m = h * k % t
            if imag:
                if m == 0 or 2 * m == t:
                    continue
                terms.append((h, -1.0, False) if 4 * m == t else (h, 1.0, False) if 4 * m == 3 * t else (h, -sn[m], True))
            else:
                if 4 * m == t or 4 * m == 3 * t:
                    continue
                terms.append((h, 1.0, False) if m == 0 else (h, -1.0, False) if 2 * m == t else (h, cs[m], True))
        s = np.zeros(v.shape[:2], np.longdouble)
        for i, (h, coeff, product) in enumerate(terms):
            s = s + v[:, :, h] * coeff
            last = i == len(terms) - 1
            if not (last and product):
                s = s.astype(np.float32)
            # By way of fp64: from extended precision NumPy rounds to fp32 first.
            s = s.astype(np.float64).astype(np.float16) if last else s.astype(np.longdouble)
        planes.append(s)
    return np.stack(planes)


@pytest.mark.parametrize("t", [3, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16])
def test_fp16_spectra_are_rounded_once(t):
    """The spectrum that eqlinear_fwd_train leaves (first dy's section, then x's: units of eight rows
    [k-step][plane][half][channel], channels padded to 64), bit for bit."""
    n, c, d = 4096, 40, 3
    g = np.random.default_rng(t)
    x = g.standard_normal((n, c * t)).astype(np.float16)
    w = dev(g.standard_normal((d, c, t)).astype(np.float16))
    wp = scratch(eql.eqlinear_packed_weight_bytes(d, c, t, eql.EQL_F16))
    eql.eqlinear_pack_weight(w, wp, d, c, t, eql.EQL_F16, eql.EQL_PACK_FWD)
    nbytes = eql.eqlinear_bwd_w_workspace_bytes(n, c, d, t, eql.EQL_F16)
    ws, y = scratch(nbytes), torch.empty((n, d * t), dtype=torch.float16, device=DEV)
    eql.eqlinear_fwd_train(dev(x), wp, y, ws, nbytes, n, c, d, t, eql.EQL_F16)
    section = (n // 16) * t * 2 * 64 * 16
    units = ws.cpu().numpy()[section:2 * section].view(np.float16).reshape(n // 16, t, 2, 64, 8)
    got = units[:, :, :, :c].transpose(1, 0, 2, 4, 3).reshape(t, n, c)
    want = plain_spectrum_f16(x, t)
    assert np.array_equal(got, want), "%d of %d values differ" % ((got != want).sum(), got.size)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", [(232, 22, 804, 4), (1000, 64, 300, 3), (197, 40, 500, 1), (60, 100, 90, 6), (900, 130, 70, 8)], ids=str)
def test_weight_gradient_with_more_workspace(shape, dtype):
    """More row ranges where the workspace holds their partial sums: the same gradient, and nothing
    written past the bytes that were given."""
    n, c, d, t = shape
    g = np.random.default_rng(n + c)
    codes, scale = B.pack(g.standard_normal((n, c * t)))
    dy = g.standard_normal((n, d * t)).astype(NP[dtype])
    ref = B.bwd_w(B.unpack(codes, scale, c * t), dy, t)
    need, room = eql.eqlinear_bwd_w_workspace_bytes(n, c, d, t, DT[dtype]), 256
    for more in (0, 256, 300000, 1 << 20, 32 << 20):
        print("case", shape, dtype, more, flush=True)
        ws = torch.full((need + more + room,), 85, dtype=torch.uint8, device=DEV)
        dw = dev(np.zeros((d, c, t), NP[dtype]))
        eql.eqlinear_bwd_w_ckpt8(dev(B.buffer(codes, scale)), None, None, eql.EQL_ACT_NONE, dev(dy), dw, ws, need + more, n, c, d, t, DT[dtype])
        got = dw.cpu().numpy().astype(np.float64)
        assert np.linalg.norm(got - ref) <= (1e-5 if dtype == "f32" else 3e-3) * np.linalg.norm(ref)
        assert (ws[need + more:] == 85).all().item()
