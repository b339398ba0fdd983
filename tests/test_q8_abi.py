"""Checks of include/eqlinear_rmsnorm.h and include/eqlinear_q8.h that need no GPU: the exports, the
sizes, and the refusals (every call below fails validation or is a no-op, so no pointer is
dereferenced)."""
import os
import re

import pytest

import group_circulant_linear_p4_amd as eql

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
P = [0x10000 + 0x10000 * i for i in range(12)]  # aligned addresses, never dereferenced
MIS = 0x10008
F16, F32, GELU, NONE = eql.EQL_F16, eql.EQL_F32, eql.EQL_ACT_GELU, eql.EQL_ACT_NONE
BIG = 1 << 40


def raw(fn, *args):
    return getattr(eql.lib(), fn)(*args)


@pytest.mark.parametrize("header,count", [("eqlinear_rmsnorm.h", 4), ("eqlinear_q8.h", 7)])
def test_exports_and_version(header, count):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(eqlinear_\w+)\s*\(", text)))
    assert len(names) == count
    for n in names:
        assert hasattr(eql.lib(), n) and hasattr(eql, n) and n in eql.__all__
    assert eql.eqlinear_rmsnorm_abi_version() == 100 and eql.eqlinear_q8_abi_version() == 100


def test_sizes():
    assert eql.eqlinear_q8_rows_bytes(0, 4, 4) == 0
    assert eql.eqlinear_q8_rows_bytes(1, 1, 1) == 16 + 4
    assert eql.eqlinear_q8_rows_bytes(5, 16, 4) == 5 * (64 + 12)
    assert eql.eqlinear_q8_rows_bytes(5, 17, 3) == 5 * (96 + 8)
    assert eql.eqlinear_q8_rows_bytes(65536, 1024, 4) == 65536 * (4096 + 12)
    assert eql.eqlinear_q8_weight_bytes(1, 1, 1) == 2048 + 32 * 4
    assert eql.eqlinear_q8_weight_bytes(1024, 1024, 4) == 1024 * (4096 + 12)
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, 0), (4, 4, 17), (4, BIG, 4), (4, 65537, 1)):
        assert eql.eqlinear_q8_rows_bytes(*bad) == 0
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 4, 17), (4, BIG, 4), (BIG, 4, 4), (4, 65537, 1)):
        assert eql.eqlinear_q8_weight_bytes(*bad) == 0


def rms_fwd(x=P[0], res=P[1], gamma=P[2], sum=P[3], y=P[4], rstd=P[5], N=8, C=4, T=4, eps=1e-5, dt=F16):
    return raw("eqlinear_rmsnorm_fwd", x, res, gamma, sum, y, rstd, N, C, T, eps, dt, None)


def test_rmsnorm_forward_refusals():
    for kw in ({"dt": 9}, {"T": 0}, {"N": -1}, {"C": 0}, {"C": BIG}, {"N": BIG}, {"x": None}, {"y": None}, {"y": P[3]},
               {"eps": -1e-9}, {"eps": float("nan")}, {"eps": float("inf")}, {"N": 1 << 22, "C": 16385, "T": 1}):
        assert rms_fwd(**kw) == eql.EQL_EINVAL, kw
    assert rms_fwd(T=17) == eql.EQL_EUNSUPPORTED
    for kw in ({"x": MIS}, {"y": MIS}, {"res": MIS}, {"sum": MIS}, {"gamma": P[2] + 1}, {"gamma": P[2] + 2, "dt": F32},
               {"rstd": P[5] + 2}):
        assert rms_fwd(**kw) == eql.EQL_EALIGN, kw
    assert rms_fwd(x=None, y=None, N=0) == eql.EQL_OK


def rms_bwd(dy=P[0], s=P[1], rstd=P[2], gamma=P[3], dres=P[4], dx=P[5], dg=P[6], ws=P[7], nbytes=None, N=8, C=4, T=4,
            dt=F16):
    if nbytes is None:
        nbytes = eql.eqlinear_rmsnorm_bwd_workspace_bytes(N, C, T, dt)
    return raw("eqlinear_rmsnorm_bwd", dy, s, rstd, gamma, dres, dx, dg, ws, nbytes, N, C, T, dt, None)


def test_rmsnorm_backward_refusals():
    need = eql.eqlinear_rmsnorm_bwd_workspace_bytes(8, 4, 4, F16)
    assert need > 0
    for kw in ({"dt": 9}, {"T": 0}, {"N": -1}, {"C": 0}, {"C": BIG}, {"N": BIG}, {"dy": None}, {"s": None}, {"rstd": None},
               {"dx": None}, {"ws": None}, {"nbytes": need - 1}, {"N": 1 << 22, "C": 8193, "T": 1}):
        assert rms_bwd(**kw) == eql.EQL_EINVAL, kw
    # Long rows keep two sums a row in the workspace, with and without the weight's gradient.
    assert rms_bwd(C=8193, T=1, dg=None, ws=None) == eql.EQL_EINVAL
    assert rms_bwd(T=17, nbytes=0) == eql.EQL_EUNSUPPORTED
    for kw in ({"dy": MIS}, {"s": MIS}, {"dres": MIS}, {"dx": MIS}, {"ws": MIS}, {"rstd": P[2] + 2}, {"gamma": P[3] + 1},
               {"dg": P[6] + 1}, {"dg": P[6] + 2, "dt": F32}):
        assert rms_bwd(**kw) == eql.EQL_EALIGN, kw
    assert rms_bwd(dy=None, s=None, rstd=None, dx=None, dg=None, ws=None, N=0) == eql.EQL_OK


def test_rmsnorm_workspace_bytes():
    assert eql.eqlinear_rmsnorm_bwd_workspace_bytes(0, 4, 4, F16) == 0
    assert eql.eqlinear_rmsnorm_bwd_workspace_bytes(4, 4, 0, F16) == 0
    assert eql.eqlinear_rmsnorm_bwd_workspace_bytes(4, 4, 4, 5) == 0
    for n in (1, 300, 1 << 20):  # one column sum a channel where the layer norm keeps two
        ours, theirs = (getattr(eql, f)(n, 96, 4, F16) for f in ("eqlinear_rmsnorm_bwd_workspace_bytes",
                                                                "eqlinear_layernorm_bwd_workspace_bytes"))
        assert 0 < 2 * ours == theirs


def quantize(x=P[0], rows=P[1], N=8, C=4, T=4, dt=F16):
    return raw("eqlinear_q8_quantize", x, rows, N, C, T, dt, None)


def q8_norm(x=P[0], res=P[1], gamma=P[2], sum=P[3], rows=P[4], N=8, C=4, T=4, eps=1e-5, dt=F16):
    return raw("eqlinear_q8_rmsnorm", x, res, gamma, sum, rows, N, C, T, eps, dt, None)


@pytest.mark.parametrize("call", [quantize, q8_norm])
def test_row_refusals(call):
    for kw in ({"dt": 9}, {"T": 0}, {"N": -1}, {"C": 0}, {"C": BIG}, {"N": BIG}, {"x": None}, {"rows": None},
               {"N": 1 << 24, "C": 32768, "T": 4}):
        assert call(**kw) == eql.EQL_EINVAL, kw
    assert call(T=17) == eql.EQL_EUNSUPPORTED
    assert call(C=65537, T=1) == eql.EQL_EUNSUPPORTED
    for kw in ({"x": MIS}, {"rows": MIS}):
        assert call(**kw) == eql.EQL_EALIGN, kw
    assert call(x=None, rows=None, N=0) == eql.EQL_OK


def test_q8_norm_refusals():
    for eps in (-1e-9, float("nan"), float("inf")):
        assert q8_norm(eps=eps) == eql.EQL_EINVAL
    for kw in ({"res": MIS}, {"sum": MIS}, {"gamma": P[2] + 1}, {"gamma": P[2] + 2, "dt": F32}):
        assert q8_norm(**kw) == eql.EQL_EALIGN, kw


def test_pack_refusals():
    def call(w=P[0], w8=P[1], D=4, C=4, T=4, dt=F16):
        return raw("eqlinear_q8_pack_weight", w, w8, D, C, T, dt, None)
    for kw in ({"dt": 9}, {"T": 0}, {"D": 0}, {"C": 0}, {"C": BIG}, {"D": BIG}, {"D": -3}, {"w": None}, {"w8": None}):
        assert call(**kw) == eql.EQL_EINVAL, kw
    assert call(T=17) == eql.EQL_EUNSUPPORTED and call(C=65537, T=1) == eql.EQL_EUNSUPPORTED
    assert call(w=MIS) == eql.EQL_EALIGN and call(w8=MIS) == eql.EQL_EALIGN


def test_product_refusals():
    def call(rows=P[0], w8=P[1], bias=P[2], res=P[3], y=P[4], N=8, C=4, D=4, T=4, dt=F16, act=NONE):
        return raw("eqlinear_q8_fwd", rows, w8, bias, res, y, N, C, D, T, dt, act, None)
    for kw in ({"dt": 9}, {"T": 0}, {"N": -1}, {"C": 0}, {"D": 0}, {"C": BIG}, {"D": BIG}, {"N": BIG}, {"rows": None},
               {"w8": None}, {"y": None}, {"act": 2}, {"act": -1}, {"N": (1 << 31) - (1 << 20), "D": 65536}):
        assert call(**kw) == eql.EQL_EINVAL, kw
    assert call(T=17) == eql.EQL_EUNSUPPORTED and call(C=65537, T=1) == eql.EQL_EUNSUPPORTED
    for kw in ({"rows": MIS}, {"w8": MIS}, {"y": MIS}, {"res": MIS}, {"bias": P[2] + 1}, {"bias": P[2] + 2, "dt": F32}):
        assert call(**kw) == eql.EQL_EALIGN, kw
    assert call(rows=None, w8=None, y=None, N=0) == eql.EQL_OK
