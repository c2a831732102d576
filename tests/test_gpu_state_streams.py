"""A state initialised and stepped on a stream of its own, with the current stream still at work
and no synchronisation before the end: the bits of the same calls on one stream."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

SHAPES = [(96, 160), (96,), (160, 96), (160,)]


def zero1(dtype):
    return fs.Zero1State(SHAPES, 2, param_dtype=dtype)


def zero1_step(st, grads, stream):
    st.step(grads, fs.MuonHparams(lr=0.01), stream=stream)


def sharded(dtype):
    return fs.ShardedState(SHAPES, None, 2, param_dtype=dtype)


def sharded_step(st, grads, stream):
    st.step(grads, stream=stream)


def run(make, step, dtype, how):
    g, n = lu.gen(9), make(dtype).layout.info["full_numel"]
    full = (torch.randn(n, generator=g, device="cuda") * 0.05).to(dtype)
    grads = [torch.randn(n, generator=g, device="cuda").to(dtype) for _ in range(2)]
    busy, spare = torch.randn(8192, 8192, device="cuda"), torch.empty(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):                           # tens of milliseconds of work on the current stream
        torch.matmul(busy, busy, out=spare)
    stream = {"current": None, "side": side, "handle": side.cuda_stream}[how]
    st = make(dtype)
    st.init_from_full(full, stream)
    for _ in range(3):
        step(st, grads, stream)
    torch.cuda.synchronize()
    fs.fsdp_check_status()
    return {k: v for k, v in vars(st).items() if torch.is_tensor(v)} | {f"params{i}": p for i, p in enumerate(getattr(st, "params", []))}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("make,step", [pytest.param(zero1, zero1_step, id="zero1"), pytest.param(sharded, sharded_step, id="sharded")])
def test_initialised_and_stepped_on_another_stream(make, step, dtype):
    want = run(make, step, dtype, "current")
    for how in ("side", "handle"):
        got = run(make, step, dtype, how)
        assert want.keys() == got.keys() and all(torch.equal(want[k], got[k]) for k in want), how
