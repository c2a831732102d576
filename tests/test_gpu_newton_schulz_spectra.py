"""Newton-Schulz steps and the Muon step on matrices whose mass is spread unevenly: over a few
columns or rows, over parts of the products' K steps, over the diagonal, over few or decaying
singular values.  Bounds: ns_util's, which go by what fp32 products make of the same matrix."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu
import ns_util as nu
import test_gpu_muon as muon

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def noise(m, n, g):
    return torch.randn(m, n, generator=g, device="cuda")


def weak(count, of):
    """All columns but `count` are `of` times as large."""
    return lambda m, n, g: noise(m, n, g) * torch.where(torch.arange(n, device="cuda") < count, 1.0, of)


def weak_rows(m, n, g):
    return noise(m, n, g) * torch.where(torch.arange(m, device="cuda") < 4, 1.0, 1e-4)[:, None]


def every_64(first, last):
    """Mass in some columns of every K step of 64."""
    def make(m, n, g):
        c = torch.arange(n, device="cuda") % 64
        return noise(m, n, g) * torch.where((c >= first) & (c < last), 1.0, 1e-3)
    return make


def diagonal(m, n, g):
    return torch.eye(m, n, device="cuda") * (1 + 0.1 * noise(1, n, g)) + 1e-4 * noise(m, n, g)


def sparse(m, n, g):
    return noise(m, n, g) * (torch.rand(m, n, generator=g, device="cuda") < 0.01)


def spectrum(values):
    def make(m, n, g):
        k = min(m, n)
        u, v = (torch.linalg.qr(noise(r, k, g).double())[0] for r in (m, n))
        return ((u * values(k)) @ v.t()).float()
    return make


def few(k):
    return torch.where(torch.arange(k, device="cuda") < 4, 1.0, 1e-3).double()


KINDS = {"noise": noise, "one column": weak(1, 1e-4), "four columns": weak(4, 1e-4), "16 columns": weak(16, 1e-3),
         "64 columns": weak(64, 1e-2), "four rows": weak_rows, "16 of 64": every_64(0, 16), "last 16 of 64": every_64(48, 64),
         "diagonal": diagonal, "sparse": sparse, "few values": spectrum(few),
         "decay": spectrum(lambda k: torch.logspace(0, -4, k, device="cuda").double())}
SIZES = [(64, 120), (128, 400), (256, 256), (200, 6644), (5000, 150), (384, 1200), (800, 2400), (1024, 4096), (5504, 2048)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_uneven_matrices(rows, cols, kind):
    g = lu.gen(rows + cols)
    x = KINDS[kind](rows, cols, g)
    y, z = torch.empty_like(x), torch.empty(rows, cols, dtype=BF16, device="cuda")
    ws = torch.empty(fs.fsdp_newton_schulz_workspace_bytes(1, rows, cols), dtype=torch.uint8, device="cuda")
    fs.fsdp_newton_schulz(x, y, workspace=ws)
    fs.fsdp_newton_schulz(x, z, workspace=ws)
    fs.fsdp_check_status()
    nu.check(y, x, kind)
    nu.check(z, x, f"{kind}, bf16")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["four columns", "16 columns", "four rows"])
def test_muon_step_of_uneven_matrices(kind, dtype):
    """The weights that the step keeps are fp32, whatever the replicas' type."""
    shapes = [(800, 2400), (2400, 800), (192, 1000)]
    z = muon.Zero1(shapes, 2, dtype, 3, grad_dtype=F32)
    g = lu.gen(4)
    for t, (r, c) in enumerate(shapes):
        for q in range(2):
            z.part(z.grads[q], t).copy_(KINDS[kind](r, c, g).reshape(-1) * 1e-3)
        z.rows(z.momentum, t).copy_(KINDS[kind](r, c, g).reshape(-1) * 1e-3)
    hp = fs.MuonHparams(lr=0.02, momentum=0.9, nesterov=True, scale="rms")
    before = muon.snapshot(z, shapes)
    z.call([0, 1, 2], hp)
    fs.fsdp_check_status()
    for t, shape in enumerate(shapes):
        muon.expect(z, t, shape, hp, "rms", before)


# Steps of the Muon step may share a pass over X: an error of A, 2^-22 of it, grows by the square of the first
# coefficient with each of two steps that A is carried on, and comes into the polynomial times the second coefficient.
# What of it lies in small directions the last two steps multiply by that square once more; elements' roundings
# that are independent leave an error of A smaller by the root of its rows, 14 and more.
CARRIED = 2.0 ** -22 * nu.COEFFS[0] ** 4 * abs(nu.COEFFS[1])


@pytest.mark.parametrize("kind", ["one column", "four columns", "64 columns", "four rows", "decay"])
@pytest.mark.parametrize("rows,cols", [(200, 6644), (1024, 4096), (2400, 800)])
def test_update_of_uneven_matrices(rows, cols, kind):
    """The update alone: weights and momentum of zero, a step of 1."""
    z = muon.Zero1([(rows, cols)], 1, F32, 3)
    x = KINDS[kind](rows, cols, lu.gen(5))
    z.part(z.grads[0], 0).copy_(x.reshape(-1))
    z.part(z.params[0], 0).zero_()
    z.rows(z.momentum, 0).zero_()
    z.call([0], fs.MuonHparams(lr=1.0, momentum=0.0, nesterov=False, scale="none"))
    fs.fsdp_check_status()
    want, plain = nu.steps_in(x, torch.float64), nu.steps_in(x, torch.float32)
    err = float((z.part(z.params[0], 0).view(rows, cols).double() + want).norm())
    assert err <= 4 * float((plain.double() - want).norm()) + (16 * 2.0 ** -22 + CARRIED) * float(want.norm())
