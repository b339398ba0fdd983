"""Every launch of every torch layer, forward and backward, happens on its tensors' device: on a machine whose current
device is another one they would otherwise run on two devices' streams without an order between them.

No GPU needed: the launches are replaced by a record of whether the device was set, on host tensors.
"""
import pytest
import torch

import group_circulant_linear_p4_amd as eql
from group_circulant_linear_p4_amd import layer

LAUNCHES = sorted(n for n, v in vars(layer).items() if n.startswith("eqlinear_") and not n.endswith("_bytes")
                  and getattr(eql, n, None) is v)


@pytest.fixture
def record(monkeypatch):
    """Launches so far as (name, devices set around it)."""
    calls, inside = [], []

    class Device:
        def __init__(self, t):
            self.t = t

        def __enter__(self):
            inside.append(self.t.device)

        def __exit__(self, *exc):
            inside.pop()
    monkeypatch.setattr(layer, "_on_device", Device)
    for name in LAUNCHES:
        monkeypatch.setattr(layer, name, lambda *a, _name=name, **kw: calls.append((_name, tuple(inside))))
    return calls


def run_all(dtype):
    kw = {"dtype": dtype}
    x = lambda f=32: torch.randn(3, f, dtype=torch.float32).to(dtype).requires_grad_(True)  # noqa: E731

    def step(y):
        for v in y if isinstance(y, tuple) else (y,):
            v.backward(torch.ones_like(v), retain_graph=True)
    for keep in (True, False):
        step(layer.EQLinear(8, 12, 4, keep_spectra=keep, **kw)(x()))
        step(layer.EQLinear(8, 12, 4, bias=True, activation="gelu", keep_spectra=keep, **kw)(x(), x(48)))
        step(layer.EQLinearP4M(4, 5, keep_spectra=keep, **kw)(x()))
        step(layer.EQLayerNorm(8, 4, ckpt8=keep, **kw)(x()))
    step(layer.EQLinear(8, 12, 4, bias=True, **kw)(x()))
    for residual in (None, x()):
        step(layer.EQRMSNorm(8, 4, **kw)(x(), residual))
    for norm in ("layer", "rms"):
        block = layer.EQMLPBlock(8, 12, 4, norm=norm, **kw)
        step(block(x()))
        with torch.no_grad():
            layer.EQMLPBlock8bit.from_float(block)(x())
    with torch.no_grad():
        layer.EQLinear8bit.from_float(layer.EQLinearP4M(4, 5, **kw))(x())


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["f16", "f32"])
def test_launches_are_on_their_tensors_device(record, dtype):
    run_all(dtype)
    assert {name for name, _ in record} <= set(LAUNCHES)
    bare = sorted({name for name, devices in record if not devices})
    assert not bare, "launched on whatever device is the current one: %s" % ", ".join(bare)
    assert all(devices[-1] == torch.device("cpu") for _, devices in record)


def test_every_launch_is_covered(record):
    run_all(torch.float16)
    run_all(torch.float32)
    assert sorted({name for name, _ in record}) == LAUNCHES
