"""CPU checks of the block operators' edges (oracle/block_oracle.py and include/eqlinear_block.h)."""
import numpy as np
import pytest

import group_circulant_linear_p4_amd as eql
from oracle import block_oracle as B


@pytest.mark.parametrize("dtype,last", [("f16", 9), ("f32", 121)])
def test_checkpoint_of_the_largest_values(dtype, last):
    """Steps stop where 127 of them are the type's last; values stay within 1 / 127 of the block's
    largest, and one below that limit nothing changes."""
    np_type = np.float16 if dtype == "f16" else np.float32
    top = np.ldexp(127.5, last)
    x = np.zeros((4, 32), np_type)
    x[0, :3] = np.finfo(np_type).max, -np.finfo(np_type).max, np.ldexp(1.0, last + 5)
    x[1, 0] = top
    x[2, 0] = np.nextafter(np_type(top), np_type(0))
    x[3, 0] = np.ldexp(1.0, last)
    codes, scale = B.pack(x, dtype)
    assert list(scale[:, 0]) == [last + 127, last + 127, last + 127, last + 127 - 6]
    assert list(codes[0, :3]) == [127, -127, 32] and codes[1, 0] == codes[2, 0] == 127 and codes[3, 0] == 64
    with np.errstate(over="raise"):
        back = B.unpack(codes, scale, 32).astype(np_type)
    assert (np.abs(back.astype(np.float64) - x) <= np.abs(x.astype(np.float64)).max(1, keepdims=True) / 127).all()


def test_weight_gradient_workspace_is_the_plain_passes():
    """A training step holds this many bytes from forward to backward, so it is what the plain passes
    need and nothing for other entry points: spectra and one set of partial sums a row range."""
    for args, nbytes in (((197, 128, 1024, 1, 0), 626688),
                         ((1000, 1024, 512, 4, 1), 37552128),
                         ((232, 22, 804, 4, 0), 520640),
                         ((12608, 96, 384, 4, 1), 37404672),
                         ((2000, 256, 256, 4, 1), 11436032),
                         ((248, 1714, 592, 6, 0), 39589632),
                         ((473, 717, 1391, 6, 1), 37207600),
                         ((65536, 1024, 1024, 4, 1), 1207959552),
                         ((16384, 64, 64, 8, 0), 79364096),
                         ((1, 1, 1, 1, 0), 4352)):
        assert eql.eqlinear_bwd_w_workspace_bytes(*args) == nbytes, args


def test_block_sees_what_changed_in_its_submodules():
    """Whether the 8-bit path's reading of the parameters stands for calling the submodules."""
    import torch
    from group_circulant_linear_p4_amd.layer import EQLayerNorm, EQLinear, EQMLPBlock

    class Own(EQLinear):
        def forward(self, x, residual=None):
            return x

    def change(f):
        block = EQMLPBlock(3, 5, 4)
        f(block)
        return block._as_made()

    assert change(lambda b: None)
    assert change(lambda b: setattr(b, "fc1", EQLinear(3, 9, 4, bias=True, activation="gelu")))
    assert change(lambda b: b.norm.__setattr__("eps", 1e-3)) and change(lambda b: setattr(b.fc2, "activation", "none"))
    assert change(lambda b: b.fc1.register_forward_hook(print).remove())
    for name in ("norm", "fc1", "fc2"):
        for register in ("register_forward_hook", "register_forward_pre_hook", "register_full_backward_hook",
                         "register_full_backward_pre_hook"):
            assert not change(lambda b: getattr(getattr(b, name), register)(print)), (name, register)
        assert not change(lambda b: setattr(getattr(b, name), "forward", print)), name
        assert not change(lambda b: setattr(b, name, torch.nn.Identity())), name
        assert not change(lambda b: setattr(getattr(b, name), "bias", None)), name
    assert not change(lambda b: setattr(b, "fc2", Own(5, 3, 4, bias=True)))
    assert not change(lambda b: setattr(b, "norm", EQLayerNorm(6, 2)))
    assert not change(lambda b: setattr(b.fc1, "activation", None)) and not change(lambda b: setattr(b.fc2, "activation", "gelu"))
