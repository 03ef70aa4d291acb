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


class _Tensor:
    """Stands for a contiguous tensor of CUDA device `index`."""

    is_cuda = True

    def __init__(self, dtype, *shape, index=0):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), index

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def _head_calls():
    """(call, its arguments by name): every tensor that it takes among them."""
    F, H, I = torch.float32, torch.bfloat16, torch.int32
    Q, S, B = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8
    t = _Tensor
    status, room = t(I, 1), t(B, 1 << 20)
    off, slots = t(I, 4), t(I, 5, 2)
    p8 = dict(xs=t(Q, 10, 48), xs_scales=t(S, 10, 4), offsets=off, weight=t(Q, 3, 24, 48),
              weight_scales=t(S, 3, 24, 4), in_features=40, d_status=status)
    yield gs.gs_layer_norm_fwd, dict(x=t(H, 5, 8), weight=t(F, 8), bias=t(F, 8), out=t(H, 5, 8))
    yield gs.gs_layer_norm_bwd, dict(grad_y=t(H, 5, 8), x=t(H, 5, 8), weight=t(F, 8), mean=t(F, 5),
                                     rstd=t(F, 5), out=t(H, 5, 8), workspace=room)
    yield gs.gs_expert_sort, dict(expert_ids=slots, experts=3, workspace=room)
    yield gs.gs_expert_dispatch, dict(x=t(H, 5, 8), slots=slots, offsets=off, d_status=status,
                                      out=t(H, 10, 8))
    yield gs.gs_expert_combine, dict(ys=t(H, 10, 8), slots=slots, weights=t(F, 5, 2),
                                     d_status=status, out=t(H, 5, 8))
    yield gs.gs_expert_combine_bwd, dict(grad_y=t(H, 5, 8), ys=t(H, 10, 8), slots=slots,
                                         weights=t(F, 5, 2), offsets=off, d_status=status)
    yield gs.gs_expert_linear_fwd, dict(xs=t(H, 10, 8), offsets=off, weight=t(H, 3, 16, 8),
                                        bias=t(H, 3, 16), d_status=status, out=t(H, 10, 16),
                                        workspace=room)
    yield gs.gs_expert_linear_bwd, dict(grad_ys=t(H, 10, 16), xs=t(H, 10, 8), offsets=off,
                                        weight=t(H, 3, 16, 8), d_status=status, workspace=room)
    yield gs.gs_expert_route_fwd, dict(logits=t(F, 5, 6), topk=2, keep=t(torch.bool, 5),
                                       workspace=room)
    yield gs.gs_expert_route_bwd, dict(logits=t(F, 5, 6), ids=slots, counts=t(I, 7),
                                       grad_weights=t(F, 5, 2), grad_loss=t(F, 1),
                                       d_status=status, out=t(F, 5, 6))
    yield gs.gs_rows_pack8, dict(x=t(F, 10, 40))
    yield gs.gs_rows_unpack8, dict(q=p8["xs"], scales=p8["xs_scales"], channels=40, dtype=H,
                                   out=t(H, 10, 40))
    yield gs.gs_expert_linear8_fwd, dict(p8, bias=t(H, 3, 24), dtype=H, out=t(H, 10, 24))
    yield gs.gs_expert_linear8_bwd, dict(p8, grad_ys=t(H, 10, 24), workspace=room)


@pytest.mark.parametrize("call", list(_head_calls()), ids=lambda c: c[0].__name__)
def test_every_tensor_of_a_call_is_on_the_current_device(call, monkeypatch):
    """A pointer into another device's memory would be read or written there."""
    fn, args = call
    launched = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace_size"):
                return lambda *_: 256
            return lambda *_: launched.append(name) or 0

    monkeypatch.setattr(gs, "lib", Library)
    monkeypatch.setattr(gs, "_new", lambda shape, dtype, *_: _Tensor(dtype, *shape))
    monkeypatch.setattr(gs, "_raw_stream", lambda device: 70 + device)
    monkeypatch.setattr(gs, "_devices", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    fn(**args)
    assert launched == [fn.__name__]
    for name, value in args.items():
        if not isinstance(value, _Tensor):
            continue
        elsewhere = _Tensor(value.dtype, *value.shape, index=1)
        with pytest.raises(ValueError, match="device"):
            fn(**{**args, name: elsewhere})
    assert launched == [fn.__name__]


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
