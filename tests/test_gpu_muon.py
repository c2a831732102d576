"""The ZeRO-1 Muon step against its definition in 64 bits."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu
import ns_util as nu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


class Zero1:
    """The buffers of a ZeRO-1 layout: N replicas, N gradients, owner rows with NaN in their gaps."""

    def __init__(self, shapes, ranks, dtype, seed, grad_dtype=None, units=None):
        g = lu.gen(seed)
        self.L = L = fs.Layout(shapes, units, n_ranks=ranks, mode=fs.FSDP_ZERO1)
        P = L.info["numel"]
        full = torch.randn(P, generator=g, device="cuda") * 0.05
        self.params = [full.to(dtype) for _ in range(ranks)]
        self.grads = [torch.empty(P, dtype=grad_dtype or dtype, device="cuda") for _ in range(ranks)]
        self.momentum = torch.full((ranks, L.stride), float("nan"), device="cuda")
        self.master = torch.full((ranks, L.stride), float("nan"), device="cuda") if dtype == BF16 else None
        for t, sh in enumerate(shapes):
            n, at = L.tensor(t)["numel"], L.tensor(t)["full_off"]
            for q in range(ranks):
                v = nu.gradient(sh[0], n // sh[0], g) if len(sh) > 1 else torch.randn(n, generator=g, device="cuda") * 1e-3
                self.grads[q][at:at + n] = v.reshape(-1).to(self.grads[q].dtype)
            self.rows(self.momentum, t).copy_(torch.randn(n, generator=g, device="cuda") * 1e-3)
            if self.master is not None:
                self.rows(self.master, t).copy_(full[at:at + n])

    def rows(self, buf, t):
        d = self.L.tensor(t)
        return buf[self.L.owner(t), d["shard_off"]:d["shard_off"] + d["numel"]]

    def part(self, full, t):
        d = self.L.tensor(t)
        return full[d["full_off"]:d["full_off"] + d["numel"]]

    def workspace(self, tensors):
        n = fs.fsdp_zero1_muon_workspace_bytes(self.L, tensors)
        return torch.full((n // 4,), float("nan"), device="cuda")

    def call(self, tensors, hp, workspace=None, **k):
        fs.fsdp_zero1_muon_broadcast(self.L, tensors, self.grads, self.master, self.momentum, self.params, hp,
                                     workspace=self.workspace(tensors) if workspace is None else workspace, **k)


def scale64(kind, rows, cols):
    return {"none": 1.0, "shape": max(1.0, rows / cols) ** 0.5, "rms": 0.2 * max(rows, cols) ** 0.5}[kind]


def expect(z, t, shape, hp, scale, before, coeffs=None):
    """Compares one tensor's momentum, weights and replicas with the definition."""
    rows, cols = shape[0], z.L.tensor(t)["numel"] // shape[0]
    beta, om = float(hp.momentum), 1.0 - float(hp.momentum)
    g = sum(z.part(q, t).double() for q in z.grads) / z.L.N
    mag = sum(z.part(q, t).double().abs() for q in z.grads) / z.L.N
    m = beta * before["momentum"][t].double() + om * g
    # the replicas' sum and mean round N + 1 times, the products and sums after them four
    lu.check(z.rows(z.momentum, t), m, U * ((z.L.N + 4) * om * mag + 3 * m.abs()), "momentum")
    u = beta * z.rows(z.momentum, t).double() + om * g if hp.nesterov else z.rows(z.momentum, t).double()
    u = u.view(rows, cols)
    k = dict(steps=hp.steps, coeffs=coeffs, eps=hp.eps)
    o64, o32 = nu.steps_in(u, torch.float64, **k), nu.steps_in(u, torch.float32, **k)
    step = float(hp.lr) * scale64(scale, rows, cols)
    w0 = before["weight"][t].double().view(rows, cols)
    w = (1.0 - float(hp.lr) * float(hp.weight_decay)) * w0 - step * o64
    got = z.rows(z.master, t) if z.master is not None else z.part(z.params[0], t)
    size = float(o64.norm())
    # the orthogonalised update's bound (ns_util), the update's own roundings, N + 4 of 2^-24, times the
    # slope of its singular values, below 4 on average over a spectrum that fills [0.68, 1.21], and
    # the weights' four roundings
    tol = step * (4 * float((o32.double() - o64).norm()) + (16 * 2.0 ** -22 + 4 * (z.L.N + 4) * U) * size) + 4 * U * float(w.norm())
    assert float((got.double().view(rows, cols) - w).norm()) <= tol
    for p in z.params:
        assert torch.equal(z.part(p, t), got.to(p.dtype))


def snapshot(z, shapes):
    return {"momentum": [z.rows(z.momentum, t).clone() for t in range(len(shapes))],
            "weight": [(z.rows(z.master, t) if z.master is not None else z.part(z.params[0], t)).clone() for t in range(len(shapes))],
            "params": z.params[0].clone(), "all": [b.clone() for b in (z.momentum, z.master) if b is not None]}


SHAPES = [(64, 32), (64,), (32, 64), (32,), (7, 5), (1, 130), (3, 8, 10), (300, 257), (257,), (129, 33), (33, 129), (64, 32)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ranks,nesterov,scale,decay", [(1, True, "rms", 0.0), (3, False, "shape", 0.1), (4, True, "none", 0.01),
                                                        (8, False, "rms", 0.5)])
def test_step(dtype, ranks, nesterov, scale, decay):
    z = Zero1(SHAPES, ranks, dtype, ranks)
    tensors = [t for t, s in enumerate(SHAPES) if len(s) > 1 and t != 9]         # one matrix is left out too
    hp = fs.MuonHparams(lr=0.02, momentum=0.9, weight_decay=decay, nesterov=nesterov, scale=scale)
    before = snapshot(z, SHAPES)
    ws = z.workspace(tensors)
    z.call(tensors, hp, ws)
    fs.fsdp_check_status()
    for t in tensors:
        expect(z, t, SHAPES[t], hp, scale, before)
    # the other tensors, and the gaps between the owner rows' tensors, are as they were
    for t in set(range(len(SHAPES))) - set(tensors):
        assert torch.equal(z.rows(z.momentum, t), before["momentum"][t])
        for p in z.params:
            assert torch.equal(z.part(p, t), z.part(before["params"], t))
    for buf, old in zip([b for b in (z.momentum, z.master) if b is not None], before["all"]):
        assert torch.equal(buf.isnan(), old.isnan())


@pytest.mark.parametrize("param,grad", [(BF16, F32), (F32, BF16)])
def test_gradient_type_of_its_own(param, grad):
    shapes = [(96, 200), (11,), (200, 96)]
    z = Zero1(shapes, 2, param, 3, grad)
    hp, before = fs.MuonHparams(lr=0.01, momentum=0.95, scale="none"), snapshot(z, shapes)
    z.call([2, 0], hp)
    for t in (0, 2):
        expect(z, t, shapes[t], hp, "none", before)


def test_schedule_of_its_own():
    shapes = [(96, 200)]
    z = Zero1(shapes, 2, F32, 4)
    coeffs = [(15 / 8, -10 / 8, 3 / 8)] * 3
    hp, before = fs.MuonHparams(lr=0.01, steps=3, scale="rms"), snapshot(z, shapes)
    z.call([0], hp, coeffs=coeffs)
    expect(z, 0, shapes[0], hp, "rms", before, coeffs)


def test_order_and_neighbours_do_not_matter():
    """The tensors' order, and a batch that passes in parts, change no bits; a second call gives them again."""
    shapes = [(40, 56)] * 70 + [(56, 40)]
    hp = fs.MuonHparams()
    z, y = Zero1(shapes, 2, BF16, 5), Zero1(shapes, 2, BF16, 5)
    z.call(list(range(71)), hp)
    y.call(list(reversed(range(71))), hp)
    assert all(torch.equal(a, b) for a, b in zip(z.params, y.params))
    assert torch.equal(z.momentum.nan_to_num(7.0), y.momentum.nan_to_num(7.0))


def test_beside_adamw():
    """One step of a layout whose matrices take Muon and whose vectors, in a unit of their own, AdamW."""
    shapes, units = [(64, 48), (48, 64), (64,), (48,)], [0, 0, 1, 1]
    z = Zero1(shapes, 2, BF16, 6, units=units)
    sq, hp = torch.zeros_like(z.momentum), fs.MuonHparams(lr=0.02)
    before = snapshot(z, shapes)
    z.call([0, 1], hp)
    fs.fsdp_zero1_adamw_broadcast(z.L, 1, 2, z.grads, z.master, z.momentum, sq, z.params, (1e-2, 0.9, 0.999, 1e-8, 0.0), 1)
    fs.fsdp_check_status()
    for t in (0, 1):
        expect(z, t, shapes[t], hp, "rms", before)
    for t in (2, 3):
        g = sum(z.part(q, t).double() for q in z.grads) / 2
        m = 0.9 * before["momentum"][t].double() + 0.1 * g
        w = before["weight"][t].double() - 1e-2 * (m / 0.1) / ((g * g).sqrt() + 1e-8)
        assert ((z.rows(z.master, t).double() - w).abs() <= 1e-5 * (w.abs() + 1)).all()


def test_captured_and_replayed():
    shapes = [(200, 120), (7,), (120, 200)]
    z, y = Zero1(shapes, 2, BF16, 7), Zero1(shapes, 2, BF16, 7)
    hp, ws = fs.MuonHparams(), z.workspace([0, 2])
    Zero1(shapes, 2, BF16, 7).call([0, 2], hp, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.call([0, 2], hp, ws)
    for k in range(3):
        for a, b in zip(z.grads, y.grads):
            a.mul_(1.0 - 0.25 * k)
            b.copy_(a)
        graph.replay()
        y.call([0, 2], hp)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(z.params, y.params))
    assert torch.equal(z.master.nan_to_num(7.0), y.master.nan_to_num(7.0))
    fs.fsdp_check_status()


def test_nothing_listed():
    z = Zero1([(8, 8)], 1, F32, 8)
    old = z.params[0].clone()
    z.call([], fs.MuonHparams(), torch.empty(0, device="cuda"))
    assert torch.equal(z.params[0], old)
