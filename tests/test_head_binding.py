"""The binding's own checks of the feature-head calls, without a GPU."""

import pytest
import torch

from tile_gaussian_splat_gb300 import binding as gs


class _On:
    """Stands for a tensor of CUDA device `index`, or a stream on it."""

    is_cuda = True
    cuda_stream = 5

    def __init__(self, index):
        self.index = self.device_index = index

    def get_device(self):
        return self.index


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device, whose memory the tensors
    have to be in; so does the stream."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(gs, "_raw_stream", lambda device: 70 + device)
    assert gs._on(None, _On(0)) == 70 and gs._on(_On(0), _On(0)) == 5
    for stream, tensor in ((None, _On(1)), (_On(1), _On(1)), (_On(1), _On(0))):
        with pytest.raises(ValueError, match="device"):
            gs._on(stream, tensor)
