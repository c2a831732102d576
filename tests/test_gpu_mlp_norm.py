"""ResidualMLP with a layer norm in front of its blocks, Zero1State, and the training example's ways
through both, as they are used together."""
import os
import sys

import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EPS = 1e-5


def reference(mlp, params, x, step, row0):
    """The blocks in 64 bits from their definition; params and x may require gradients."""
    for b in range(mlp.blocks):
        w1, b1, w2, b2, g, c = params[6 * b:6 * b + 6]
        d = x - x.mean(1, keepdim=True)
        n = d * (d.square().mean(1, keepdim=True) + EPS) ** -0.5 * g + c
        s = torch.nn.functional.gelu(n @ w1.t() + b1) @ w2.t() + b2
        if mlp.p:
            spec = fs.DropoutSpec(mlp.p, mlp.seed, step * mlp.blocks + b, row0)
            s = torch.where(lu.keep_mask(*s.shape, spec), s / (1 - mlp.p), torch.zeros_like(s))
        x = x + s
    return x


def build(width, hidden, p, seed=0):
    mlp = fs.ResidualMLP(width, hidden, 2, p=p, seed=99, norm=True, eps=EPS)
    layout = fs.Layout(*mlp.shapes(), 3, fs.FSDP_FLAT)
    full, g = torch.zeros(layout.info["full_numel"], device="cuda"), lu.gen(seed)
    mlp.initialise(layout, full, g)
    for v in fs.tensor_views(layout, full):
        if v.dim() == 1:
            v += torch.randn(v.shape, generator=g, device="cuda") * 0.1
    return mlp, layout, full, g


# widths whose views start at odd elements of the full buffer, and aligned ones
@pytest.mark.parametrize("width,hidden,rows", [(48, 96, 40), (37, 65, 21)])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_gradients_against_autograd(width, hidden, rows, p):
    mlp, layout, full, g = build(width, hidden, p)
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
    # six fp32 layers deep, each within some 1e-6 of its result (in norm)
    for got, w, what in [(y, y64, "y"), (dx, want[0], "dx")] + [
            (a, b, f"param {t}") for t, (a, b) in enumerate(zip(fs.tensor_views(layout, grad), want[1:]))]:
        assert (got.double() - w).norm() <= 1.5e-5 * w.norm(), what


def test_gradient_against_differences():
    """The directional derivative of the loss against central differences of the same forward
    (steps as in the test without norm)."""
    mlp, layout, full, g = build(48, 96, 0.2)
    x, dy = (torch.randn(64, 48, generator=g, device="cuda") for _ in range(2))
    grad = torch.zeros_like(full)
    mlp.forward(layout, full, x, 1)
    mlp.backward(layout, full, grad, dy, 1)
    for t in range(12):
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
    mlp, layout, full, g = build(48, 96, 0.1)
    x, dy = (torch.randn(96, 48, generator=g, device="cuda") for _ in range(2))
    whole, parts = torch.zeros_like(full), torch.zeros_like(full)
    mlp.forward(layout, full, x, 2)
    mlp.backward(layout, full, whole, dy, 2)
    for k, r in enumerate(range(0, 96, 32)):
        mlp.forward(layout, full, x[r:r + 32], 2, row0=r)
        mlp.backward(layout, full, parts, dy[r:r + 32], 2, row0=r, accumulate=k > 0)
    assert (whole - parts).norm() <= 1e-5 * whole.norm()


def test_passes_on_two_streams():
    """Forward on one stream and backward on another, beside a second pair: the bits of a pass alone."""
    mlp, layout, full, g = build(64, 128, 0.1)
    x, dy = (torch.randn(200, 64, generator=g, device="cuda") for _ in range(2))
    want, dx = torch.zeros_like(full), None
    mlp.forward(layout, full, x, 1)
    dx = mlp.backward(layout, full, want, dy, 1)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        got = torch.zeros_like(full)
        a.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(a):
            mlp.forward(layout, full, x, 1)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            out = mlp.backward(layout, full, got, dy, 1)
        with torch.cuda.stream(a):
            torch.randn(200, 64, device="cuda")           # takes freed memory on forward's stream
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(out, dx)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zero1_state_is_its_calls(dtype):
    """A step of Zero1State against the calls that it stands for, bit for bit."""
    mlp = fs.ResidualMLP(40, 72, 2, norm=True)
    shapes, _ = mlp.shapes()
    st = fs.Zero1State(shapes, 3, param_dtype=dtype)
    assert st.muon == [0, 2, 6, 8] and len(st.adamw_units) == 4
    full, g = torch.zeros(st.layout.info["full_numel"], device="cuda"), lu.gen(4)
    mlp.initialise(st.layout, full, g)
    st.init_from_full(full.to(dtype))
    L, master = st.layout, None if st.master is None else st.master.clone()
    m, v, params = torch.zeros_like(st.exp_avg), torch.zeros_like(st.exp_avg), [p.clone() for p in st.params]
    hp, adamw = fs.MuonHparams(lr=0.01), (2e-3, 0.9, 0.99, 1e-8, 0.1)
    ws = torch.empty(fs.fsdp_zero1_muon_workspace_bytes(L, st.muon), dtype=torch.uint8, device="cuda")
    for step in (1, 2):
        grads = [torch.randn(full.numel(), generator=g, device="cuda") * 1e-3 for _ in range(3)]
        st.step(grads, hp, adamw)
        fs.fsdp_zero1_muon_broadcast(L, st.muon, grads, master, m, params, hp, ws)
        for u in st.adamw_units:
            fs.fsdp_zero1_adamw_broadcast(L, u, u + 1, grads, master, m, v, params, adamw, step)
    assert all(torch.equal(a, b) for a, b in zip(st.params, params)) and torch.equal(st.exp_avg, m) and torch.equal(st.exp_avg_sq, v)
    assert master is None or torch.equal(master, st.master)
    assert all(torch.equal(p, st.params[0]) for p in st.params)


@pytest.mark.parametrize("dtype,optimizer,micro", [(torch.bfloat16, "muon", 2), (torch.float32, "muon", 1), (torch.bfloat16, "adamw", 1)])
def test_training_example_runs(dtype, optimizer, micro):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_mlp
    losses = train_mlp.train(width=64, hidden=256, blocks=2, ranks=3, rows=128, micro=micro, steps=6, p=0.05, dtype=dtype,
                             lr=3e-3, say=lambda *a: None, norm=True, optimizer=optimizer)
    assert len(losses) == 6 and all(x == x and x < float("inf") for x in losses)


def test_zero1_state_on_another_stream():
    shapes, g = [(96, 160), (96,), (160, 96), (160,)], lu.gen(9)
    side = torch.cuda.Stream()
    out = []
    for stream in (None, side, side.cuda_stream):
        g.manual_seed(9)
        st = fs.Zero1State(shapes, 2)
        st.init_from_full((torch.randn(st.layout.info["full_numel"], generator=g, device="cuda") * 0.05).bfloat16())
        grads = [torch.randn(st.layout.info["full_numel"], generator=g, device="cuda").bfloat16() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(3):
            st.step(grads, fs.MuonHparams(lr=0.01), stream=stream)
            torch.empty(1 << 22, dtype=torch.uint8, device="cuda").fill_(255)     # what the current stream does with memory it is given
        torch.cuda.synchronize()
        out.append(st.params[1].clone())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
