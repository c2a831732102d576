"""ResidualMLP's calls and buffers, on the host: the layer calls are replaced by recorders."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs
from fsdp_sharded_state_gb300 import mlp as mlp_module


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("fsdp_linear_forward", "fsdp_linear_dgrad", "fsdp_linear_wgrad", "fsdp_dropout"):
        monkeypatch.setattr(mlp_module, name, lambda *a, _name=name, **k: seen.append((_name, a, k)))
    return seen


def build(width=24, hidden=40, blocks=2, p=0.1):
    mlp = fs.ResidualMLP(width, hidden, blocks, p=p)
    layout = fs.Layout(*mlp.shapes(), 3, fs.FSDP_FLAT)
    return mlp, layout, torch.zeros(layout.info["full_numel"])


def test_every_pass_has_scratch_of_its_own(calls):
    """Passes may run beside each other on streams of their own: no two of them get the same
    scratch (the recorder holds on to it, as work still under way does), and each call gets all
    that it may need."""
    mlp, layout, full = build()
    x = torch.zeros(7, 24)
    scratch = []
    for _ in range(2):
        calls.clear()
        mlp.forward(layout, full, x)
        scratch.append([k["workspace"] for _, _, k in calls])
        calls.clear()
        mlp.backward(layout, full, full, x)
        scratch.append([k["workspace"] for n, _, k in calls if n != "fsdp_dropout"])
    need = max(fs.fsdp_linear_workspace_bytes(7, i, o, torch.float32, False) for i, o in ((24, 40), (40, 24)))
    for one in scratch:
        assert len({w.data_ptr() for w in one}) == 1 and all(w.numel() >= need for w in one)
    assert len({one[0].data_ptr() for one in scratch}) == len(scratch)


class Kept:
    """A tensor's stand-in that notes the streams it is recorded for."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_what_forward_kept_outlives_a_backward_on_another_stream(calls, monkeypatch):
    """The caching allocator gives a freed tensor's memory out again in the order of the stream
    that it was made on; what backward reads on another one has to be recorded for it."""
    mlp, layout, full = build()
    x = torch.zeros(7, 24)
    for streams, recorded in (((1, 1), []), ((1, 2), [2])):
        monkeypatch.setattr(mlp_module, "_current_stream", lambda t: streams[0])
        mlp.forward(layout, full, x)
        mlp.saved = kept = [tuple(Kept() for _ in saved) for saved in mlp.saved]
        kept = [k for saved in kept for k in saved]
        assert len(kept) == 6
        monkeypatch.setattr(mlp_module, "_current_stream", lambda t: streams[1])
        monkeypatch.setattr(mlp_module.torch, "empty_like", lambda t: x)
        mlp.backward(layout, full, full, x)
        assert all(k.streams == recorded for k in kept)
