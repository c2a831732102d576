"""init_from_full(stream=s), on the host: every operation on the state's buffers runs with s as the
current stream, between a wait of s for the current stream and one of the current stream for s."""
import contextlib

import pytest
import torch
from torch.overrides import TorchFunctionMode

import fsdp_sharded_state_gb300 as fs
from fsdp_sharded_state_gb300 import state as state_module
from fsdp_sharded_state_gb300 import zero1 as zero1_module


class FakeStream:
    def __init__(self, name, seen):
        self.name, self.seen, self.cuda_stream = name, seen, hash(name)

    def wait_stream(self, other):
        self.seen.append((self.name, "waits for", other.name))


class Recorder(TorchFunctionMode):
    """In-place operations on tensors, with the stream that was current."""

    def __init__(self, seen, current):
        super().__init__()
        self.seen, self.current = seen, current

    def __torch_function__(self, func, types, args=(), kwargs=None):
        name = getattr(func, "__name__", "")
        if name in ("copy_", "zero_"):
            self.seen.append((name, "on", self.current[-1].name))
        return func(*args, **(kwargs or {}))


@pytest.fixture
def world(monkeypatch):
    """The events, and a side stream beside the current one, neither of a device."""
    seen = []
    current = [FakeStream("current", seen)]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    side = FakeStream("side", seen)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: side)

    def reshard(*a):
        stream = a[6] if len(a) > 6 else None
        named = "side" if stream in (side, side.cuda_stream) else current[-1].name if stream is None else "unknown"
        seen.append(("reshard", "on", named))

    for module in (state_module, zero1_module):
        monkeypatch.setattr(module, "fsdp_reshard", reshard)
    return seen, current, side


def check(make, world, operations, handle):
    seen, current, side = world
    st = make()
    full = torch.zeros(st.layout.info["full_numel"])
    with Recorder(seen, current):
        st.init_from_full(full, side.cuda_stream if handle else side)
    assert seen[0] == ("side", "waits for", "current") and seen[-1] == ("current", "waits for", "side")
    assert sorted(seen[1:-1]) == sorted((op, "on", "side") for op in operations)
    seen.clear()
    with Recorder(seen, current):
        st.init_from_full(full)
    assert sorted(seen) == sorted((op, "on", "current") for op in operations)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zero1_state(world, dtype, handle):
    operations = ["copy_"] * 2 + ["zero_"] * 2 + (["reshard"] if dtype == torch.bfloat16 else [])
    check(lambda: fs.Zero1State([(8, 4), (8,)], 2, param_dtype=dtype, device="cpu"), world, operations, handle)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sharded_state(world, dtype, handle):
    check(lambda: fs.ShardedState([(8, 4), (8,)], None, 2, param_dtype=dtype, device="cpu"), world, ["zero_"] * 2 + ["reshard"], handle)
