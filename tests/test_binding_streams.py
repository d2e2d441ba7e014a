"""The training operators' choice of device and stream, on the CPU: torch's
device and stream contexts are stood in for."""
import contextlib

import pytest
import torch

from row_wise_reduction_gb300 import rowops


class _Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its context would make that device current, and the call would end up on
    the tensors' device's own current stream, in order with nothing."""
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    ran = []
    with pytest.raises(ValueError, match="stream"):
        rowops._elsewhere(lambda: ran.append(1), _Stream(1), 0)
    assert not ran
    assert rowops._elsewhere(lambda: 7, _Stream(1), 1) == 7
    assert rowops._elsewhere(lambda: 8, None, 1) == 8
