"""Schedules of coefficients where steps share a pass over X: bf16 results and the Muon step's update, of
sizes that take groups of two and of three.  Steps differ from each other, so that a coefficient
or a scale of another step shows.

Bounds: ns_util's, and what sharing adds: an error of A, 2^-22 of it over the root of its rows (elements'
roundings are independent), grows by the square of the first coefficient with each of up to two
steps that A is carried on, comes into the polynomial times the second and third coefficient, and is multiplied by the
first coefficients of the steps that follow."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu
import ns_util as nu
import test_gpu_muon as muon

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

STRONG = [(8.28721201814563, -23.595886519098837, 17.300387312530933), (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
          (3.9486908534822946, -2.908902115962949, 0.5518191394370137)]
CUBIC, QUINTIC, STILL = (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8), (1.0, 0.0, 0.0)
USUAL = nu.COEFFS
SCHEDULES = {
    "1": [USUAL], "2": [USUAL] * 2, "3": [USUAL] * 3, "4": [USUAL] * 4, "7": [USUAL] * 7, "8": [USUAL] * 5 + [CUBIC] * 3,
    # gains of 8.3, 4.1 and 3.9 and more: a group ends between the second and the third
    "strong": STRONG, "strong, then others": STRONG + [(2.0, -0.9, 0.15), QUINTIC, CUBIC, STILL],
    # every step another polynomial, of gains that groups of three hold
    "all differ": [(2.0, -1.5, 0.5), CUBIC, QUINTIC, (1.9, -1.3, 0.4), STILL, (1.7, -0.7, 0.0), (1.2, -0.3, 0.1)],
    "strong, a step later": [STILL] + STRONG + [CUBIC],
    "one large gain": [(19.0, -76.0, 60.8), (0.25, 0.0, 0.0), CUBIC, QUINTIC],
    "nothing left": [QUINTIC, (0.0, 0.0, 0.0), CUBIC],
}
SIZES = [(173, 6644), (4000, 96), (800, 2400), (2300, 770)]


def carried(coeffs, m):
    most = 0.0
    for j, (_, b, c) in enumerate(coeffs):
        v = abs(b) + abs(c)
        for i in (j - 1, j - 2):
            v *= max(1.0, coeffs[i][0] ** 2) if i >= 0 else 1.0
        for a, _, _ in coeffs[j + 1:]:
            v *= max(1.0, abs(a))
        most = max(most, v)
    return most * 2.0 ** -22 / m ** 0.5


@pytest.mark.parametrize("name", SCHEDULES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_schedules(rows, cols, name):
    coeffs = SCHEDULES[name]
    x = nu.gradient(rows, cols, lu.gen(rows), rank=8)
    k = dict(steps=len(coeffs), coeffs=coeffs)
    y, z = torch.empty_like(x), torch.empty(rows, cols, dtype=BF16, device="cuda")
    ws = torch.empty(fs.fsdp_newton_schulz_workspace_bytes(1, rows, cols), dtype=torch.uint8, device="cuda")
    fs.fsdp_newton_schulz(x, y, workspace=ws, **k)
    fs.fsdp_newton_schulz(x, z, workspace=ws, **k)
    fs.fsdp_check_status()
    nu.check(y, x, name, **k)
    nu.check(z, x, f"{name}, bf16", **k)
    # the update of a Muon step: weights and momentum of zero, a step of 1
    s = muon.Zero1([(rows, cols)], 1, F32, 3)
    s.part(s.grads[0], 0).copy_(x.reshape(-1))
    s.part(s.params[0], 0).zero_()
    s.rows(s.momentum, 0).zero_()
    s.call([0], fs.MuonHparams(lr=1.0, momentum=0.0, nesterov=False, scale="none", steps=len(coeffs)), coeffs=coeffs)
    fs.fsdp_check_status()
    want, plain = nu.steps_in(x, torch.float64, **k), nu.steps_in(x, torch.float32, **k)
    err = float((s.part(s.params[0], 0).view(rows, cols).double() + want).norm())
    tol = 4 * float((plain.double() - want).norm()) + (16 * 2.0 ** -22 + carried(coeffs, min(rows, cols))) * float(want.norm())
    assert err <= tol
