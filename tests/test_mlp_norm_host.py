"""ResidualMLP with norm and Zero1State, on the host: shapes, units and the order of calls."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs
from fsdp_sharded_state_gb300 import mlp as mlp_module
from fsdp_sharded_state_gb300 import zero1 as zero1_module


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("fsdp_linear_forward", "fsdp_linear_dgrad", "fsdp_linear_wgrad", "fsdp_dropout", "fsdp_layernorm_forward",
                 "fsdp_layernorm_backward"):
        monkeypatch.setattr(mlp_module, name, lambda *a, _name=name, **k: seen.append((_name, a, k)))
    return seen


def test_calls_of_a_block(calls):
    mlp = fs.ResidualMLP(24, 40, 2, norm=True)
    layout = fs.Layout(*mlp.shapes(), 3, fs.FSDP_FLAT)
    assert layout.info["n_tensors"] == 12 and layout.n_units == 2
    full, x = torch.zeros(layout.info["full_numel"]), torch.zeros(7, 24)
    mlp.initialise(layout, full)
    views = fs.tensor_views(layout, full)
    assert (views[4] == 1).all() and not views[5].any() and not views[1].any() and views[0].any()
    mlp.forward(layout, full, x)
    assert [n for n, _, _ in calls] == ["fsdp_layernorm_forward", "fsdp_linear_forward", "fsdp_linear_forward"] * 2
    calls.clear()
    mlp.backward(layout, full, full, x, accumulate=True)
    assert [n for n, _, _ in calls] == ["fsdp_linear_wgrad", "fsdp_linear_dgrad", "fsdp_linear_wgrad", "fsdp_linear_dgrad",
                                        "fsdp_layernorm_backward"] * 2
    need = fs.fsdp_layernorm_workspace_bytes(7, 24)
    for n, a, k in calls:
        if n == "fsdp_layernorm_backward":
            assert k["accumulate"] and k["residual"] is not None and k["workspace"].numel() >= need
    assert mlp.saved == []


def test_without_norm_nothing_changes(calls):
    mlp = fs.ResidualMLP(24, 40, 1)
    layout = fs.Layout(*mlp.shapes(), 3, fs.FSDP_FLAT)
    full, x = torch.zeros(layout.info["full_numel"]), torch.zeros(7, 24)
    mlp.forward(layout, full, x)
    mlp.backward(layout, full, full, x)
    assert [n for n, _, _ in calls] == ["fsdp_linear_forward"] * 2 + ["fsdp_linear_wgrad", "fsdp_linear_dgrad"] * 2


def test_zero1_units(monkeypatch):
    seen = []
    monkeypatch.setattr(zero1_module, "fsdp_zero1_muon_broadcast", lambda L, t, *a, **k: seen.append(("muon", tuple(t))))
    monkeypatch.setattr(zero1_module, "fsdp_zero1_adamw_broadcast", lambda L, a, b, *r, **k: seen.append(("adamw", a, b)))
    st = fs.Zero1State([(8, 4), (8,), (4,), (4, 8), (3, 1), (2, 3, 4)], 2, device="cpu")
    assert st.muon == [0, 3] and st.layout.unit_ids == [0, 1, 1, 2, 3, 3] and st.adamw_units == [1, 3]
    st.step([torch.zeros(1)] * 2)
    assert seen == [("muon", (0, 3)), ("adamw", 1, 2), ("adamw", 3, 4)] and st.t == 1
    st = fs.Zero1State([(8, 4), (4,)], 2, muon=[], device="cpu", param_dtype=torch.float32)
    assert st.master is None and st.adamw_units == [0] and st.layout.n_units == 1
    with pytest.raises(TypeError):
        fs.Zero1State([(8, 4)], 2, param_dtype=torch.float16, device="cpu")
