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
