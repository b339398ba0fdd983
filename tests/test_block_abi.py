"""Checks of include/eqlinear_block.h that need no GPU: the exports, the sizes, and the refusals
(every call below fails validation or is a no-op, so no pointer is dereferenced)."""
import os
import re

import pytest

import group_circulant_linear_p4_amd as eql

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "eqlinear_block.h")
P = [0x10000 + 0x10000 * i for i in range(12)]  # aligned addresses, never dereferenced
MIS = 0x10008
F16, F32, GELU, NONE = eql.EQL_F16, eql.EQL_F32, eql.EQL_ACT_GELU, eql.EQL_ACT_NONE
BIG = 1 << 40


def raw(fn, *args):
    return getattr(eql.lib(), fn)(*args)


def test_exports_and_version():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(eqlinear_\w+)\s*\(", text)))
    assert len(names) == 11
    for n in names:
        assert hasattr(eql.lib(), n) and hasattr(eql, n) and n in eql.__all__
    assert eql.eqlinear_block_abi_version() == 100


def test_checkpoint_bytes():
    assert eql.eqlinear_ckpt8_bytes(0, 4, 4) == 0
    assert eql.eqlinear_ckpt8_bytes(1, 1, 1) == 33
    assert eql.eqlinear_ckpt8_bytes(5, 8, 4) == 5 * 33
    assert eql.eqlinear_ckpt8_bytes(5, 11, 3) == 5 * (64 + 2)
    assert eql.eqlinear_ckpt8_bytes(65536, 1024, 4) == 65536 * (4096 + 128)
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 4, 0), (4, 4, 17), (4, 1 << 40, 4)):
        assert eql.eqlinear_ckpt8_bytes(*bad) == 0


@pytest.mark.parametrize("fn", ["eqlinear_ckpt8_pack", "eqlinear_ckpt8_unpack"])
def test_checkpoint_copy_refusals(fn):
    assert raw(fn, P[0], P[1], 8, 4, 4, 7, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], P[1], 8, 4, 0, F16, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], P[1], 8, 4, 17, F16, None) == eql.EQL_EUNSUPPORTED
    assert raw(fn, P[0], P[1], -8, 4, 4, F16, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], P[1], 8, 0, 4, F16, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], P[1], 8, 1 << 40, 4, F16, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], P[1], 1 << 31, 4, 4, F16, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], P[1], 1 << 30, 1024, 4, F16, None) == eql.EQL_EINVAL   # too many workgroups
    assert raw(fn, None, P[1], 8, 4, 4, F16, None) == eql.EQL_EINVAL
    assert raw(fn, P[0], None, 8, 4, 4, F16, None) == eql.EQL_EINVAL
    assert raw(fn, MIS, P[1], 8, 4, 4, F16, None) == eql.EQL_EALIGN
    assert raw(fn, P[0], MIS, 8, 4, 4, F32, None) == eql.EQL_EALIGN
    assert raw(fn, None, None, 0, 4, 4, F16, None) == eql.EQL_OK


def norm_fwd(x=P[0], gamma=P[1], beta=P[2], y=P[3], ckpt=P[4], mean=P[5], rstd=P[6], N=8, C=4, T=4, eps=1e-5, dt=F16):
    return raw("eqlinear_layernorm_fwd", x, gamma, beta, y, ckpt, mean, rstd, N, C, T, eps, dt, None)


def test_norm_forward_refusals():
    for kw in ({"dt": 9}, {"T": 0}, {"N": -1}, {"C": 0}, {"C": BIG}, {"N": BIG}, {"x": None}, {"y": None},
               {"eps": -1e-9}, {"eps": float("nan")}, {"eps": float("inf")},
               {"N": 1 << 22, "C": 16385, "T": 1}):
        assert norm_fwd(**kw) == eql.EQL_EINVAL, kw
    assert norm_fwd(T=17) == eql.EQL_EUNSUPPORTED
    for kw in ({"x": MIS}, {"y": MIS}, {"ckpt": MIS}, {"gamma": P[1] + 1}, {"beta": P[2] + 2, "dt": F32},
               {"mean": P[5] + 2}, {"rstd": P[6] + 1}):
        assert norm_fwd(**kw) == eql.EQL_EALIGN, kw
    assert norm_fwd(x=None, y=None, N=0) == eql.EQL_OK


def norm_bwd(fn, dy=P[0], src=P[1], mean=P[2], rstd=P[3], gamma=P[4], dres=P[5], dx=P[6], dg=P[7], db=P[8], ws=P[9],
             nbytes=None, N=8, C=4, T=4, dt=F16):
    if nbytes is None:
        nbytes = eql.eqlinear_layernorm_bwd_workspace_bytes(N, C, T, dt)
    stats = (mean, rstd) if fn == "eqlinear_layernorm_bwd" else (rstd,)
    return raw(fn, dy, src, *stats, gamma, dres, dx, dg, db, ws, nbytes, N, C, T, dt, None)


@pytest.mark.parametrize("fn", ["eqlinear_layernorm_bwd", "eqlinear_layernorm_bwd_ckpt8"])
def test_norm_backward_refusals(fn):
    need = eql.eqlinear_layernorm_bwd_workspace_bytes(8, 4, 4, F16)
    assert need > 0
    bad = [{"dt": 9}, {"T": 0}, {"N": -1}, {"C": 0}, {"C": BIG}, {"N": BIG}, {"dy": None}, {"src": None},
           {"rstd": None}, {"dx": None}, {"ws": None}, {"nbytes": need - 1}, {"nbytes": need - 1, "dg": None},
           {"N": 1 << 22, "C": 8193, "T": 1}]
    if fn == "eqlinear_layernorm_bwd":
        bad.append({"mean": None})
    for kw in bad:
        assert norm_bwd(fn, **kw) == eql.EQL_EINVAL, kw
    # Long rows keep two sums a row in the workspace, with and without parameter gradients.
    assert norm_bwd(fn, C=8193, T=1, dg=None, db=None, ws=None) == eql.EQL_EINVAL
    assert norm_bwd(fn, T=17, nbytes=0) == eql.EQL_EUNSUPPORTED
    for kw in ({"dy": MIS}, {"src": MIS}, {"dres": MIS}, {"dx": MIS}, {"ws": MIS}, {"rstd": P[3] + 2},
               {"gamma": P[4] + 1}, {"dg": P[7] + 1}, {"db": P[8] + 2, "dt": F32}):
        assert norm_bwd(fn, **kw) == eql.EQL_EALIGN, kw
    assert norm_bwd(fn, dy=None, src=None, rstd=None, dx=None, dg=None, db=None, ws=None, N=0) == eql.EQL_OK


def test_norm_workspace_bytes():
    assert eql.eqlinear_layernorm_bwd_workspace_bytes(0, 4, 4, F16) == 0
    assert eql.eqlinear_layernorm_bwd_workspace_bytes(4, 4, 0, F16) == 0
    assert eql.eqlinear_layernorm_bwd_workspace_bytes(4, 4, 4, 5) == 0
    small, large = (eql.eqlinear_layernorm_bwd_workspace_bytes(n, 96, 4, F16) for n in (1, 1 << 20))
    assert 2 * 96 * 4 <= small < large <= 64 << 20


def test_gelu_backward_refusals():
    fn = "eqlinear_fused_epilogue_bwd_ckpt8"
    need = eql.eqlinear_fused_epilogue_bwd_workspace_bytes(300, 5, 4, F16)

    def call(dy=P[0], pre=P[1], dpre=P[2], db=P[3], ws=P[4], nbytes=need, N=300, D=5, T=4, dt=F16):
        return raw(fn, dy, pre, dpre, db, ws, nbytes, N, D, T, dt, None)
    for kw in ({"dt": 4}, {"T": 0}, {"D": 0}, {"N": -2}, {"D": BIG}, {"dy": None}, {"pre": None}, {"dpre": None},
               {"ws": None}, {"nbytes": need - 1}):
        assert call(**kw) == eql.EQL_EINVAL, kw
    assert call(T=17) == eql.EQL_EUNSUPPORTED
    for kw in ({"dy": MIS}, {"pre": MIS}, {"dpre": MIS}, {"ws": MIS}, {"db": P[3] + 1}):
        assert call(**kw) == eql.EQL_EALIGN, kw
    assert call(dy=None, pre=None, dpre=None, db=None, ws=None, N=0) == eql.EQL_OK


def test_weight_gradient_refusals():
    need = eql.eqlinear_bwd_w_workspace_bytes(64, 4, 4, 4, F16)

    def call(ck=P[0], g=P[1], b=P[2], act=GELU, dy=P[3], dw=P[4], ws=P[5], nbytes=need, N=64, C=4, D=4, T=4, dt=F16):
        return raw("eqlinear_bwd_w_ckpt8", ck, g, b, act, dy, dw, ws, nbytes, N, C, D, T, dt, None)
    for kw in ({"dt": 4}, {"T": 0}, {"D": 0}, {"C": 0}, {"N": -2}, {"act": 2}, {"act": -1}, {"ck": None}, {"dy": None},
               {"dw": None}, {"ws": None}, {"nbytes": need - 1}):
        assert call(**kw) == eql.EQL_EINVAL, kw
    assert call(T=17) == eql.EQL_EUNSUPPORTED
    for kw in ({"ck": MIS}, {"g": P[1] + 1}, {"b": P[2] + 1}, {"dy": MIS}, {"dw": MIS}, {"ws": MIS}):
        assert call(**kw) == eql.EQL_EALIGN, kw

    def spectrum(ck=P[0], g=P[1], b=P[2], act=NONE, ws=P[5], nbytes=need, N=64, T=4, dt=F16):
        return raw("eqlinear_ckpt8_spectrum", ck, g, b, act, ws, nbytes, N, 4, 4, T, dt, None)
    for kw in ({"dt": 4}, {"T": 0}, {"N": -2}, {"act": 5}, {"ck": None}, {"ws": None}, {"nbytes": need - 1}):
        assert spectrum(**kw) == eql.EQL_EINVAL, kw
    for kw in ({"ck": MIS}, {"ws": MIS}, {"g": P[1] + 1}, {"b": P[2] + 2, "dt": F32, "nbytes": 1 << 30}):
        assert spectrum(**kw) == eql.EQL_EALIGN, kw
    assert spectrum(ck=None, ws=None, N=0) == eql.EQL_OK


def test_binding_raises_and_refuses_host_tensors():
    import torch
    with pytest.raises(eql.EqlError) as e:
        eql.eqlinear_ckpt8_pack(MIS, P[1], 8, 4, 4, F16, stream=0)
    assert e.value.status == eql.EQL_EALIGN and "eqlinear_ckpt8_pack" in str(e.value)
    with pytest.raises(ValueError):
        eql.eqlinear_layernorm_fwd(torch.zeros(8, 16), None, None, P[1], None, None, None, 8, 4, 4, 1e-5, F32, stream=0)


@pytest.mark.parametrize("what", ["weight", "bias", "dtype", "features"])
def test_layer_norm_layer_refuses(what):
    """Refused before any buffer reaches the library (CPU tensors: nothing is launched)."""
    import torch
    from group_circulant_linear_p4_amd.layer import eq_layer_norm
    x, g, b, t = torch.zeros(5, 12), torch.ones(3), torch.zeros(3), 4
    if what == "weight":
        g = torch.ones(12)
    elif what == "bias":
        b = torch.zeros(1, 3)
    elif what == "dtype":
        g = g.half()
    else:
        t = 5
    with pytest.raises(ValueError, match="features" if what == "features" else "weight" if what != "bias" else "bias"):
        eq_layer_norm(x, g, b, t)


@pytest.mark.parametrize("what", ["w2", "x", "b1", "dtype"])
def test_mlp_block_refuses(what):
    import torch
    from group_circulant_linear_p4_amd.layer import EQMLPBlock
    block = EQMLPBlock(3, 5, 4)
    x = torch.zeros(2, 12)
    if what == "w2":
        block.fc2.weight = torch.nn.Parameter(torch.zeros(3, 4, 4))
    elif what == "x":
        x = torch.zeros(2, 16)
    elif what == "b1":
        block.fc1.bias = torch.nn.Parameter(torch.zeros(20))
    else:
        x = x.half()
    with pytest.raises(ValueError, match={"w2": "w2", "x": "features", "b1": "b1", "dtype": "dtype"}[what]):
        block(x)
