"""The binding's own checks of the feature-head calls, without a GPU."""

import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from tile_gaussian_splat_gb300 import binding as gs
from tile_gaussian_splat_gb300 import build


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


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """A block that the current stream freed may still be in use there, so a
    call on another stream takes none of those; and the caller may go on with
    the result on the current stream."""
    now = ["current"]
    log = []

    class Tensor:
        def __init__(self, stream):
            self.stream = stream

        def record_stream(self, stream):
            log.append((self.stream, stream))

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.saved, now[0] = now[0], self.stream

        def __exit__(self, *_):
            now[0] = self.saved

    class Side:
        cuda_stream = 99

    like, side = _On(0), Side()
    like.device = "cuda:0"
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Tensor(now[0]))
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: now[0])
    monkeypatch.setattr(gs, "_raw_stream", lambda device: 7)
    assert gs._new((3,), torch.uint8, like, side).stream is side
    assert now == ["current"] and log == [(side, "current")]
    side.cuda_stream = 7  # the current stream itself
    assert gs._new((3,), torch.uint8, like, side).stream == "current" and len(log) == 1
    assert gs._new((3,), torch.uint8, like, None).stream == "current"


def test_imports_where_torch_has_no_cuda():
    """Sizes and argument checks need no GPU, nor a torch built for one."""
    build.build()
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda')]:\n"
            "    delattr(torch._C, name)\n"
            "from tile_gaussian_splat_gb300 import binding\n"
            "assert binding.gs_tile_bits(4, 4) == 4\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, capture_output=True)
