"""The training operators' binding refuses a stream of another device than the
tensors': the launch would go to that device."""

import pytest
import torch

from sparse_moe_layer_03_amd import train as T


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        def __init__(self, device):
            self.device, self.cuda_stream = torch.device(device), 64

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    here, calls = torch.device("cuda:0"), []
    with pytest.raises(ValueError, match="stream: on cuda:1, needed on cuda:0"):
        T._on(here, calls.append, Stream("cuda:1"))
    assert not calls
    T._on(here, calls.append, Stream("cuda:0"))
    assert [c.value for c in calls] == [64]
