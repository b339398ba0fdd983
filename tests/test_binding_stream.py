"""The binding's way to torch's current stream (no GPU needed)."""
import os

import torch

import group_circulant_linear_p4_amd as eql


def test_a_forked_process_asks_torch_again(monkeypatch):
    """The short way skips torch's check that this process may use the GPU: a child made by fork must not inherit it."""
    monkeypatch.setattr(eql, "_raw_stream", lambda: 1234)
    assert eql._stream(None) == 1234
    pid = os.fork()
    if pid == 0:
        os._exit(0 if eql._raw_stream is None else 1)
    assert os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]) == 0
    assert eql._stream(None) == 1234


def test_the_short_way_is_taken_only_once_torch_is_up(monkeypatch):
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(eql, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    assert eql._stream(None) == 77 and eql._raw_stream is None
