"""ResidualMLP on several streams at once."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu


def build(width, hidden, dtype, blocks=2):
    mlp = fs.ResidualMLP(width, hidden, blocks, act="gelu", p=0.1, seed=5)
    layout = fs.Layout(*mlp.shapes(), 3, fs.FSDP_FLAT)
    full = torch.zeros(layout.info["full_numel"], dtype=dtype, device="cuda")
    g = lu.gen(71)
    for v in fs.tensor_views(layout, full):
        v.copy_(torch.randn(v.shape, generator=g, device="cuda") * (v.shape[-1] ** -0.5 if v.dim() == 2 else 0.1))
    return mlp, layout, full, g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_passes_beside_each_other(dtype):
    """Widths whose operands are copied or split in scratch; each stream's passes against the
    same passes alone, bit for bit."""
    mlp, layout, full, g = build(257, 1021, dtype)
    xs = [(torch.randn(700, 257, generator=g, device="cuda")).to(dtype) for _ in range(3)]
    dys = [(torch.randn(700, 257, generator=g, device="cuda")).to(dtype) for _ in range(3)]

    def passes(x, dy, grad):
        y = mlp.forward(layout, full, x, 1)
        return y, mlp.backward(layout, full, grad, dy, 1), grad

    want = [passes(x, dy, torch.zeros_like(full)) for x, dy in zip(xs, dys)]
    grads = [torch.zeros_like(full) for _ in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for s, x, dy, grad in zip(streams, xs, dys, grads):
            with torch.cuda.stream(s):
                got.append(passes(x, dy, grad))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)
    fs.fsdp_check_status()


def test_forward_on_one_stream_backward_on_another():
    """What forward kept is read by a backward that another stream gets to late, while the first
    stream allocates and fills new tensors of the same sizes."""
    mlp, layout, full, g = build(256, 1024, torch.bfloat16)
    x, dy = ((torch.randn(700, 256, generator=g, device="cuda")).bfloat16() for _ in range(2))
    want, grad = torch.zeros_like(full), torch.zeros_like(full)
    mlp.forward(layout, full, x, 1)
    mlp.backward(layout, full, want, dy, 1)
    busy = torch.randn(8192, 8192, device="cuda").bfloat16()
    torch.cuda.synchronize()
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(first):
        mlp.forward(layout, full, x, 1)
    second.wait_stream(first)
    with torch.cuda.stream(second):
        for _ in range(20):
            busy @ busy
        mlp.backward(layout, full, grad, dy, 1)
    with torch.cuda.stream(first):
        for n in (256, 1024):
            for _ in range(6):
                torch.full((700, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    fs.fsdp_check_status()
    assert torch.equal(grad, want)
