"""The binding's checks of where its tensors lie, with stand-ins for tensors of two GPUs."""
import math

import pytest
import torch

import fsdp_sharded_state_gb300 as fs

BF16 = torch.bfloat16


class Tensor:
    """What the binding asks of a contiguous tensor; its address is never read."""

    def __init__(self, *shape, device=0, dtype=BF16):
        self.shape, self.device_index, self.dtype = torch.Size(shape), device, dtype
        self.is_cuda = device >= 0

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        s = tuple(math.prod(self.shape[k + 1:]) for k in range(len(self.shape)))
        return s if d is None else s[d]

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return 2

    def is_contiguous(self):
        return True


@pytest.fixture(autouse=True)
def on_the_first_gpu(monkeypatch):
    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(fs, "lib", Library)
    monkeypatch.setattr(fs, "_stream", lambda *a: None)


def tensors(call, **elsewhere):
    """Arguments of a call on the first GPU, those named in `elsewhere` on another device."""
    shapes = {"forward": dict(x=(4, 16), w=(32, 16), y=(4, 32), bias=(32,), preact=(4, 32), residual=(4, 32), workspace=(64,)),
              "dgrad": dict(dz=(4, 32), w=(32, 16), dx=(4, 16), preact=(4, 16), residual=(4, 16), workspace=(64,)),
              "wgrad": dict(dz=(4, 32), x=(4, 16), dw=(32, 16), db=(32,), workspace=(64,)),
              "dropout": dict(x=(4, 16), y=(4, 16), residual=(4, 16))}[call]
    return {k: Tensor(*s, device=elsewhere.get(k, 0)) for k, s in shapes.items()}


CALLS = {"forward": lambda **k: fs.fsdp_linear_forward(**k, act="gelu"), "dgrad": lambda **k: fs.fsdp_linear_dgrad(**k, act="gelu"),
         "wgrad": fs.fsdp_linear_wgrad, "dropout": lambda **k: fs.fsdp_dropout(**k, dropout=None)}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_one_device(call):
    CALLS[call](**tensors(call))


@pytest.mark.parametrize("where,text", [(1, "cuda:1"), (-1, "CUDA")])
@pytest.mark.parametrize("call,name", [(c, n) for c in sorted(CALLS) for n in tensors(c)])
def test_a_tensor_elsewhere_is_refused(call, name, where, text):
    with pytest.raises(ValueError, match=f"{name} is .*{text}"):
        CALLS[call](**tensors(call, **{name: where}))


@pytest.mark.parametrize("call", sorted(CALLS))
def test_tensors_of_a_gpu_that_is_not_current_are_refused(call):
    with pytest.raises(ValueError, match="current device"):
        CALLS[call](**{k: Tensor(*t.shape, device=1) for k, t in tensors(call).items()})


def test_stream_handle_without_the_private_call(monkeypatch):
    """The current stream's handle, where torch does not offer it without a Stream object."""
    monkeypatch.undo()

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(fs, "_raw_stream", None, raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    assert fs._stream(None) == 77 and fs._stream(None, 0) == 77 and fs._stream(Stream) == 77 and fs._stream(5) == 5
