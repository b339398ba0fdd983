"""GELU in the 8-bit product's epilogue (include/eqlinear_q8.h) over its whole range, against 64 bits.

With a weight of zeros the product is exactly the bias, so each output is GELU of a known value.

Bound.  v Phi(v) = max(v, 0) - |v| Q(|v|), Q = 1 - Phi, with Q = 2^p for a polynomial p that is fitted up to |v| = 5.6.
There |v| Q is off by at most 6e-5 of it and 1.4e-7 (7.9e-8 the fit; p's rounding, two steps of 2^-24 |p|, times ln 2 |v| Q
and p at most 3 where |v| Q is not small: 3e-8; the exponential's one step and the coefficients' rounding 3e-8).  Beyond 5.6, where it
is below 6e-8, it lies between 0 and the value.  The last operation rounds to fp32, and the result is rounded once
to its type: half a step each.
"""
import numpy as np
import pytest
import torch
from scipy.special import erfc

import group_circulant_linear_p4_amd as eql

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NP = {"f16": np.float16, "f32": np.float32}
TORCH = {"f16": torch.float16, "f32": torch.float32}
ULP = {"f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "f32": 2.0 ** -126}


def gelu_bound(v, dtype):
    """(GELU, how far off it may be) of values in 64 bits."""
    a = np.abs(v)
    tail = a * 0.5 * erfc(a / np.sqrt(2.0))  # |v| Q(|v|)
    ref = np.maximum(v, 0.0) - tail
    ref = np.where(v < 0, -tail, ref)
    slack = np.where(a <= 5.6, np.minimum(6e-5 * tail, 1.4e-7), tail)
    return ref, (1 + ULP[dtype]) * (slack + 2.0 ** -24 * np.abs(ref)) + ULP[dtype] * np.abs(ref) + TINY[dtype]


def inputs(dtype):
    if dtype == "f16":  # every value up to 16 in magnitude
        bits = np.arange(0x4C01, dtype=np.uint16)
        v = bits.view(np.float16)
        return np.concatenate([v, -v])
    g = np.random.default_rng(1)
    v = np.concatenate([np.linspace(-16, 16, 20001), np.linspace(-6, -3, 6001), g.standard_normal(8000), 1e-3 * g.standard_normal(500)])
    return v.astype(np.float32)


# Rows, the outputs taken at a time, T: the kernel for few rows, the small tiles, the large ones, with and without the
# residual's addition.
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n,d,t", [(1, 20000, 1), (5, 16000, 1), (70, 20000, 1), (4, 20000, 4), (20, 8000, 4), (600, 2000, 4), (40, 20000, 5)])
@pytest.mark.parametrize("residual", [False, True])
def test_gelu(n, d, t, residual, dtype):
    v = inputs(dtype)
    w8 = torch.zeros(eql.eqlinear_q8_weight_bytes(d, 1, t), dtype=torch.uint8, device=DEV)
    rows8 = torch.zeros(eql.eqlinear_q8_rows_bytes(n, 1, t), dtype=torch.uint8, device=DEV)
    eql.eqlinear_q8_quantize(torch.ones(n, t, dtype=TORCH[dtype], device=DEV), rows8, n, 1, t, TORCH[dtype])
    eql.eqlinear_q8_pack_weight(torch.zeros(d, 1, t, dtype=TORCH[dtype], device=DEV), w8, d, 1, t, TORCH[dtype])
    y = torch.zeros(n, d * t, dtype=TORCH[dtype], device=DEV)
    zeros = torch.zeros_like(y) if residual else None  # adds nothing
    for lo in range(0, len(v), d):
        bias = np.zeros(d, NP[dtype])
        part = v[lo:lo + d]
        bias[:len(part)] = part
        eql.eqlinear_q8_fwd(rows8, w8, torch.from_numpy(bias).to(DEV), zeros, y, n, 1, d, t, TORCH[dtype], eql.EQL_ACT_GELU)
        got = y.reshape(n, d, t)
        assert torch.equal(got, got[:1, :, :1].expand(n, d, t))  # every row and group element alike
        got = got[0, :len(part), 0].cpu().numpy().astype(np.float64)
        ref, bound = gelu_bound(part.astype(np.float64), dtype)
        err = np.abs(got - ref)
        at = int((err / bound).argmax())
        assert (err <= bound).all(), "GELU(%r) = %r, exactly %.9g: off by %.3g times the bound" % (
            float(part[at]), float(got[at]), ref[at], (err / bound)[at])


def test_gelu_special_values():
    """Infinities and NaN: GELU(inf) = inf, GELU(-inf) = 0, a NaN stays one."""
    bias = torch.tensor([np.inf, -np.inf, np.nan, 60000.0, -60000.0, 0.0], dtype=torch.float16, device=DEV)
    for n in (1, 40):
        w8 = torch.zeros(eql.eqlinear_q8_weight_bytes(6, 1, 1), dtype=torch.uint8, device=DEV)
        rows8 = torch.zeros(eql.eqlinear_q8_rows_bytes(n, 1, 1), dtype=torch.uint8, device=DEV)
        y = torch.empty(n, 6, dtype=torch.float16, device=DEV)
        eql.eqlinear_q8_fwd(rows8, w8, bias, None, y, n, 1, 6, 1, torch.float16, eql.EQL_ACT_GELU)
        got = y.cpu().numpy().astype(np.float64)
        assert np.isnan(got[:, 2]).all()
        assert np.array_equal(np.delete(got, 2, 1), np.broadcast_to([np.inf, 0.0, 60000.0, 0.0, 0.0], (n, 5)))
