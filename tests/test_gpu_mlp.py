"""ResidualMLP over a ShardedState's buffers: gradients against autograd in 64 bits and
against differences of the loss, and the training example."""
import os
import sys

import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def reference(mlp, params, x, step, row0):
    """The blocks in 64 bits from their definition; params and x may require gradients."""
    for b in range(mlp.blocks):
        w1, b1, w2, b2 = params[4 * b:4 * b + 4]
        z = x @ w1.t() + b1
        h = {"gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu, "relu": torch.relu}[mlp.act](z)
        s = h @ w2.t() + b2
        if mlp.p:
            spec = fs.DropoutSpec(mlp.p, mlp.seed, step * mlp.blocks + b, row0)
            s = torch.where(lu.keep_mask(*s.shape, spec), s / (1 - mlp.p), torch.zeros_like(s))
        x = x + s
    return x


def build(width, hidden, act, p, seed=0):
    mlp = fs.ResidualMLP(width, hidden, 2, act=act, p=p, seed=99)
    shapes, units = mlp.shapes()
    layout = fs.Layout(shapes, units, 3, fs.FSDP_FLAT)
    full = torch.zeros(layout.info["full_numel"], device="cuda")
    g = lu.gen(seed)
    for v in fs.tensor_views(layout, full):
        v.copy_(torch.randn(v.shape, generator=g, device="cuda") * (v.shape[-1] ** -0.5 if v.dim() == 2 else 0.1))
    return mlp, layout, full, g


# widths whose views start at odd elements of the full buffer, and aligned ones
@pytest.mark.parametrize("width,hidden,rows", [(48, 96, 40), (37, 65, 21)])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_gradients_against_autograd(width, hidden, rows, act, p):
    mlp, layout, full, g = build(width, hidden, act, p)
    x = torch.randn(rows, width, generator=g, device="cuda")
    dy = torch.randn(rows, width, generator=g, device="cuda")
    grad = torch.full((layout.info["full_numel"],), float("nan"), device="cuda")
    y = mlp.forward(layout, full, x, step=3, row0=11)
    dx = mlp.backward(layout, full, grad, dy, step=3, row0=11)
    fs.fsdp_check_status()
    params = [v.double().requires_grad_() for v in fs.tensor_views(layout, full)]
    x64 = x.double().requires_grad_()
    y64 = reference(mlp, params, x64, 3, 11)
    want = torch.autograd.grad(y64, [x64] + params, dy.double())
    # four fp32 layers deep, each within some 1e-6 of its result (in norm); relu may switch
    # where a pre-activation is within rounding of 0, which these few values do not meet
    for got, w, what in [(y, y64, "y"), (dx, want[0], "dx")] + [
            (a, b, f"param {t}") for t, (a, b) in enumerate(zip(fs.tensor_views(layout, grad), want[1:]))]:
        assert (got.double() - w).norm() <= 1e-5 * w.norm(), what


def test_gradient_against_differences():
    """The directional derivative of the loss against central differences of the same
    forward: in 32 bits, at steps where the difference's truncation (h^2) and rounding
    (2^-22 / h) are both below 1e-3."""
    mlp, layout, full, g = build(48, 96, "gelu", 0.2)
    x = torch.randn(64, 48, generator=g, device="cuda")
    dy = torch.randn(64, 48, generator=g, device="cuda")
    grad = torch.zeros_like(full)
    mlp.forward(layout, full, x, 1)
    mlp.backward(layout, full, grad, dy, 1)
    for t in range(8):
        d = torch.zeros_like(full)
        v = fs.tensor_views(layout, d)[t]
        v.copy_(torch.randn(v.shape, generator=g, device="cuda") * (v.shape[-1] ** -0.5 if v.dim() == 2 else 0.1))
        h = 2.0 ** -8
        f = [(mlp.forward(layout, full + s * h * d, x, 1).double() * dy.double()).sum() for s in (1, -1)]
        want = (f[0] - f[1]) / (2 * h)
        got = (fs.tensor_views(layout, grad)[t].double() * v.double()).sum()
        scale = (grad.double().abs() * d.double().abs()).sum()
        assert abs(got - want) <= 2e-3 * scale, t
    mlp.saved = []


def test_accumulated_micro_batches_add_up():
    mlp, layout, full, g = build(48, 96, "gelu", 0.1)
    x = torch.randn(96, 48, generator=g, device="cuda")
    dy = torch.randn(96, 48, generator=g, device="cuda")
    whole, parts = torch.zeros_like(full), torch.zeros_like(full)
    mlp.forward(layout, full, x, 2)
    mlp.backward(layout, full, whole, dy, 2)
    for k, r in enumerate(range(0, 96, 32)):
        mlp.forward(layout, full, x[r:r + 32], 2, row0=r)
        mlp.backward(layout, full, parts, dy[r:r + 32], 2, row0=r, accumulate=k > 0)
    assert (whole - parts).norm() <= 1e-5 * whole.norm()


@pytest.mark.parametrize("dtype,micro", [(torch.bfloat16, 2), (torch.float32, 1)])
def test_training_example_learns(dtype, micro):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_mlp
    losses = train_mlp.train(width=64, hidden=256, blocks=2, ranks=3, rows=128, micro=micro, steps=25, p=0.05, dtype=dtype,
                             lr=3e-3, say=lambda *a: None)
    assert losses[-1] < 0.6 * losses[0]
