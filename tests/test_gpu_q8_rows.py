"""The 8-bit row kernels (include/eqlinear_q8.h) in every arrangement of lanes that the number of rows and the row's
length select, for every group order, against the fp64 definition (oracle/q8_oracle.py).

Each batch repeats BASE rows: those are checked against the definition, the others to be the same bits.

Bounds, derived from the formulas.
  * A plane is a sum of T products in fp32, within (T + 2) 2^-24 of the sum of magnitudes (the norm's weight another
    rounding); times 127 / m (two roundings) and to an integer: a code is within half of the fp64 plane's times 127 / m,
    plus that error times 127 / m, plus 127 * 2^-22.  At T = 1, 2 and 4 the planes of these inputs are exact, and the codes equal.
  * A scale is m / 127 rounded to nearest, 2^-24 of it; through the norm times 1 / rms: the sum of squares adds at most 16
    values a chunk in a chain and joins at most 10 times (half of the 26 roundings' 2^-24, as a root), its mean, the root and the
    product another five: 18 * 2^-24, below 2^-19.
"""
import numpy as np
import pytest
import torch

import group_circulant_linear_p4_amd as eql
from oracle import q8_oracle as Q

DEV = "cuda:0"
NP = {"f16": np.float16, "f32": np.float32}
TORCH = {"f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
BASE = 37


def chunk(t, elt):
    """Channels that a lane takes at a time."""
    if elt == 2:
        return {1: 16, 2: 8, 3: 4, 4: 4}.get(t, 1)
    return {1: 8, 2: 4}.get(t, 1)


def arrangement(c, t, elt, n):
    """(lanes, chunks a lane) of the row kernels; 0 chunks: the row is read twice."""
    chunks, values = -(-c // chunk(t, elt)), chunk(t, elt) * t
    some = 1 if n <= 1024 else next((k for k in (4, 2) if 32 // values >= k), 1)
    keep = 8 if 64 // values >= 8 else 4
    lanes = 16 if n > 4096 and chunks <= 16 * some else (64 if chunks <= 64 * some else 256)
    k = -(-chunks // lanes)
    return lanes, 0 if k > keep else next(s for s in (1, 2, 4, 8) if s >= k)


def cases(t, elt):
    """A (rows, channels) for each arrangement that any can select, the last chunk a ragged one."""
    ch, found = chunk(t, elt), {}
    for n in (3, 1030, 4099):
        for chunks in (3, 16, 27, 59, 64, 101, 190, 256, 500, 1000, 2000, 2100):
            c = chunks * ch - (ch // 2 if ch > 1 else 0)
            if n > 3 and c * t > 6000:
                continue
            found.setdefault(arrangement(c, t, elt, n), (n, c))
    return found


def test_every_arrangement_is_tested():
    for elt in (2, 4):
        for t in range(1, 17):
            values = chunk(t, elt) * t
            some = next((k for k in (4, 2) if 32 // values >= k), 1)
            want = {(16, 1), (64, 1), (256, 1), (256, 2), (256, 4), (256, 0)}
            want |= {(lanes, k) for lanes in (16, 64) for k in (2, 4) if k <= some}
            want |= {(256, 8)} if 64 // values >= 8 else set()
            assert set(cases(t, elt)) == want, (t, elt)


def values(n, c, t, dtype, seed):
    g = np.random.default_rng([seed, n, c, t])
    # Multiples of 2^-6 below 16: exact in fp16, and any sums of them in fp32.
    v = np.round(g.standard_normal((n, c, t)) * 2.0 ** 6) * 2.0 ** -6 + 0.25
    return v.astype(NP[dtype])


def on_gpu(a, n):
    a = torch.from_numpy(np.ascontiguousarray(a.reshape(a.shape[0], -1))).to(DEV)
    return a.repeat(-(-n // a.shape[0]), 1)[:n].contiguous()


def first_rows(buf, n, c, t):
    """The first BASE rows' codes and scales, after the others were compared with them."""
    pitch, f, m = -(-c // 16) * 16, t // 2 + 1, min(n, BASE)
    codes, scales = buf[:n * t * pitch].reshape(n, -1), buf[n * t * pitch:n * t * pitch + 4 * n * f].reshape(n, -1)
    at = torch.arange(n, device=DEV) % BASE
    assert torch.equal(codes, codes[at]) and torch.equal(scales, scales[at])
    part = torch.cat([codes[:m].reshape(-1), scales[:m].reshape(-1)]).cpu().numpy()
    codes, scales, pad = Q.read_rows(part, m, c, t)
    assert not pad.any()
    return codes, scales


def check(codes, scales, pl, mags, t, off, dtype):
    """Codes and scales against the planes pl [T, rows, C]: exact codes at T = 1, 2 and 4 (pl then in fp32)."""
    rc, rs = Q.encode(pl, t)
    for f, where in enumerate(Q.frequencies(t)[1]):
        if t in (1, 2, 4):
            assert np.array_equal(codes[where], rc[where])
            assert (np.abs(scales[:, f] - rs[:, f]) <= off * rs[:, f]).all()
            continue
        m = np.maximum(np.abs(pl[where]).max((0, 2)), Q.FLOOR)
        err = (t + 4) * 2.0 ** -24 * mags.max(1)
        assert (np.abs(scales[:, f] * 127.0 - m) <= err + off * m).all()
        want = pl[where] * (127.0 / m)[:, None]
        slack = 0.5 + 127.0 * (2.0 ** -22 + (2 * err / m)[:, None])
        assert (np.abs(codes[where].astype(np.float64) - want) <= slack).all()
        assert np.abs(codes[where].astype(int)).max() <= 127


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("t", range(1, 17))
def test_quantize_arrangements(t, dtype):
    for shape, (n, c) in cases(t, 2 if dtype == "f16" else 4).items():
        print("case q8 rows", t, dtype, shape, n, c, flush=True)
        x = values(min(n, BASE), c, t, dtype, 0)
        buf = torch.full((eql.eqlinear_q8_rows_bytes(n, c, t),), 0xFF, dtype=torch.uint8, device=DEV)
        eql.eqlinear_q8_quantize(on_gpu(x, n), buf, n, c, t, TORCH[dtype])
        check(*first_rows(buf, n, c, t), Q.planes(x, t), np.abs(x.astype(np.float64)).sum(2), t, 2.0 ** -23, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("t", range(1, 17))
def test_norm_arrangements(t, dtype):
    for shape, (n, c) in cases(t, 2 if dtype == "f16" else 4).items():
        print("case q8 norm", t, dtype, shape, n, c, flush=True)
        x, r = values(min(n, BASE), c, t, dtype, 1), values(min(n, BASE), c, t, dtype, 2)
        gamma = (1 + 0.2 * np.random.default_rng(5).standard_normal(c)).astype(NP[dtype])
        kept = (x.astype(np.float64) + r.astype(np.float64)).astype(NP[dtype])
        xd, gd = on_gpu(x, n), torch.from_numpy(gamma).to(DEV)
        buf = torch.full((eql.eqlinear_q8_rows_bytes(n, c, t),), 0xFF, dtype=torch.uint8, device=DEV)
        eql.eqlinear_q8_rmsnorm(xd, on_gpu(r, n), gd, xd, buf, n, c, t, EPS, TORCH[dtype])  # the sum in x's place
        assert torch.equal(xd, on_gpu(kept, n))
        codes, scales = first_rows(buf, n, c, t)
        k64, g64 = kept.astype(np.float64), gamma.astype(np.float64)
        rstd = Q.rmsnorm(kept.reshape(len(kept), -1), None, t, EPS)[2]
        pl = Q.planes(k64, t) * g64[None, None]
        if t in (1, 2, 4):  # exact in fp32 before the weight, times it rounded once
            pl = (Q.planes(k64, t).astype(np.float32) * gamma.astype(np.float32)[None, None]).astype(np.float64)
        check(codes, scales / rstd[:, None], pl, np.abs(k64).sum(2) * np.abs(g64), t, 2.0 ** -19 + 2.0 ** -23, dtype)
        without = torch.full_like(buf, 0xFF)
        eql.eqlinear_q8_rmsnorm(on_gpu(kept, n), None, gd, None, without, n, c, t, EPS, TORCH[dtype])
        assert torch.equal(without, buf)
