"""A row's 8-bit form and its outputs are the same bits alone and in a batch of any size (include/eqlinear_q8.h),
through every arrangement of lanes and every product kernel that the number of rows selects.

Inputs are rows of general values, so a sum of squares taken in another order is another float for one row in
five or so; every batch repeats the same BASE rows.  Exact comparisons: no tolerance.
"""
import numpy as np
import pytest
import torch

import group_circulant_linear_p4_amd as eql

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "f32": torch.float32}
BASE = 64


def normal(shape, seed, dtype):
    v = np.random.default_rng([seed, *shape]).standard_normal(shape) * 1.3 + 0.1
    return torch.from_numpy(v.astype(np.float32)).to(DEV).to(TORCH[dtype])


def repeated(base, n):
    return base.repeat(-(-n // BASE), 1)[:n].contiguous()


def split_rows(buf, n, c, t):
    """(codes [n, T, pitch], scales [n, F]) of 8-bit rows, on the GPU."""
    pitch, f = -(-c // 16) * 16, t // 2 + 1
    codes = buf[:n * t * pitch].reshape(n, t, pitch)
    return codes, buf[n * t * pitch:n * t * pitch + 4 * n * f].view(torch.float32).reshape(n, f)


def norm_rows(base, res, gamma, n, c, t, dtype):
    buf = torch.zeros(eql.eqlinear_q8_rows_bytes(n, c, t), dtype=torch.uint8, device=DEV)
    eql.eqlinear_q8_rmsnorm(repeated(base, n), repeated(res, n), gamma, None, buf, n, c, t, 1e-6, TORCH[dtype])
    return split_rows(buf, n, c, t)


# (C, T): what a row is spread over changes at 1024 and 4096 rows.  The comments give (lanes, chunks a lane) up to 1024
# rows, from 1025 and from 4097: fp16; fp32.
CHANGING = [(40, 3),    # (64, 1), (64, 1), (16, 1); (64, 1), (64, 1), (16, 4)
            (96, 4),    # (64, 1), (64, 1), (16, 2); (256, 1), (64, 2), (64, 2)
            (512, 4),   # (256, 1), (64, 2), (64, 2); (256, 2)
            (60, 5),    # (64, 1), (64, 1), (16, 4) in both
            (133, 5),   # (256, 1), (64, 4), (64, 4) in both
            (64, 8),    # (64, 1), (64, 1), (16, 4) in both
            (1024, 1),  # (64, 1); (256, 1), (64, 2), (64, 2)
            (2000, 1),  # (256, 1), (64, 2), (64, 2); (256, 1), (64, 4), (64, 4)
            (30, 16),   # (64, 1), (64, 1), (16, 2) in both
            (700, 4)]   # (256, 1); (256, 4)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("shape", CHANGING, ids=str)
def test_norm_rows_in_batches(shape, dtype):
    c, t = shape
    base, res, gamma = normal((BASE, c * t), 1, dtype), normal((BASE, c * t), 2, dtype), normal((c,), 3, dtype)
    codes, scales = norm_rows(base, res, gamma, BASE, c, t, dtype)
    for n in (1, 3, 1024, 1025, 4096, 4097):
        print("case q8 norm rows", shape, dtype, n, flush=True)
        got_codes, got_scales = norm_rows(base, res, gamma, n, c, t, dtype)
        at = torch.arange(n, device=DEV) % BASE
        assert torch.equal(got_codes, codes[at])
        assert torch.equal(got_scales, scales[at]), "%d of %d rows' scales differ" % (
            int((got_scales != scales[at]).any(1).sum()), n)


def product_rows(base, w8, bias, res, n, c, d, t, act, dtype):
    rows8 = torch.zeros(eql.eqlinear_q8_rows_bytes(n, c, t), dtype=torch.uint8, device=DEV)
    eql.eqlinear_q8_quantize(repeated(base, n), rows8, n, c, t, TORCH[dtype])
    y = torch.empty(n, d * t, dtype=TORCH[dtype], device=DEV)
    eql.eqlinear_q8_fwd(rows8, w8, bias, None if res is None else repeated(res, n), y, n, c, d, t, TORCH[dtype], act)
    return y


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("t", range(1, 17))
def test_outputs_in_batches(t, dtype):
    """The kernel for few rows, the small tiles, and both of the large ones (12 group elements and fewer)."""
    c, d, sizes = (460, 140, (1, 3, 40, 4200, 33000 if t == 1 else 16500)) if t <= 2 else (36, 40, (1, 4, 40, 4200, 12300))
    base, w, bias = normal((BASE, c * t), 4, dtype), normal((d, c, t), 5, dtype), normal((d,), 6, dtype)
    res = normal((BASE, d * t), 7, dtype)
    w8 = torch.zeros(eql.eqlinear_q8_weight_bytes(d, c, t), dtype=torch.uint8, device=DEV)
    eql.eqlinear_q8_pack_weight(w, w8, d, c, t, TORCH[dtype])
    for act in (eql.EQL_ACT_NONE, eql.EQL_ACT_GELU):
        for r in (None, res):
            want = product_rows(base, w8, bias, r, BASE, c, d, t, act, dtype)
            for n in sizes:
                print("case q8 outputs", t, dtype, act, r is not None, n, flush=True)
                got = product_rows(base, w8, bias, r, n, c, d, t, act, dtype)
                assert torch.equal(got, want[torch.arange(n, device=DEV) % BASE])
