"""Calls on tensors of another device than the current one run on theirs (no GPU needed)."""
import torch

from group_circulant_linear_p4_amd import layer


class _Tensor:
    def __init__(self, is_cuda, index):
        self.is_cuda, self.device = is_cuda, torch.device("cuda", index) if is_cuda else torch.device("cpu")


def test_launch_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    other = layer._on_device(_Tensor(True, 1))
    assert isinstance(other, torch.cuda.device) and other.idx == 1
    assert layer._on_device(_Tensor(True, 0)) is layer._HERE
    with layer._on_device(_Tensor(False, 0)):  # host tensors go on to the call, which refuses them
        pass
