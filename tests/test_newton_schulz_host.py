"""Argument checks of Newton-Schulz and of the Muon step, on the host: every call below carries
exactly one invalid argument, so it is refused before any CUDA call."""
import ctypes as C

import pytest
import torch

import fsdp_sharded_state_gb300 as fs

P = 1 << 20                                     # an aligned address that nothing reads
EINVAL, EDTYPE, ESHAPE, EALIGN, EOVERFLOW = -1, -2, -3, -4, -5
NAN, INF = float("nan"), float("inf")


def arr(t, v):
    return None if v is None else (t * max(1, len(v)))(*v)


def ns(**k):
    a = dict(count=2, rows=8, cols=16, src=(P, P), lds=(16, 16), sdt=0, dst=(P, P), ldd=(16, 16), ddt=0, steps=5, coeffs=None,
             eps=1e-7, ws=P, nws=1 << 30)
    a.update(k)
    return fs.lib().fsdp_newton_schulz(a["count"], a["rows"], a["cols"], arr(C.c_void_p, a["src"]), arr(C.c_int64, a["lds"]), a["sdt"],
                                       arr(C.c_void_p, a["dst"]), arr(C.c_int64, a["ldd"]), a["ddt"], a["steps"],
                                       arr(C.c_float, a["coeffs"]), a["eps"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(count=-1), ESHAPE), (dict(rows=0), ESHAPE), (dict(cols=0), ESHAPE), (dict(rows=(1 << 20) + 1), EOVERFLOW),
    (dict(rows=1 << 18, cols=1 << 17, lds=(1 << 17,) * 2, ldd=(1 << 17,) * 2), EOVERFLOW),
    (dict(sdt=2), EDTYPE), (dict(ddt=-1), EDTYPE), (dict(steps=0), EINVAL), (dict(steps=65), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=9e-17), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL), (dict(src=None), EINVAL), (dict(dst=None), EINVAL),
    (dict(lds=None), EINVAL), (dict(ldd=None), EINVAL), (dict(src=(P, None)), EINVAL), (dict(dst=(None, P)), EINVAL),
    (dict(src=(P, P + 2)), EALIGN), (dict(ddt=1, dst=(P + 1, P)), EALIGN), (dict(lds=(16, 15)), ESHAPE), (dict(ldd=(15, 16)), ESHAPE),
    (dict(lds=(16, 1 << 32)), EOVERFLOW), (dict(ws=None), EINVAL), (dict(nws=1000), EINVAL), (dict(ws=P + 8), EALIGN),
    (dict(steps=1, coeffs=(NAN, 0, 0)), EINVAL), (dict(steps=1, coeffs=(4.5, 0, 0)), EINVAL),           # reaches 4.5 at s = 1
    (dict(steps=2, coeffs=(3, 0, 0, 2, 0, 0)), EINVAL),                                                 # 6 after two steps
    (dict(steps=1, coeffs=(12, -11, 0)), EINVAL),                                                       # 1 at s = 1, 4.8 inside
    (dict(steps=1, coeffs=(2000, -4e6, 2e9)), EINVAL),
])
def test_refused(bad, status):
    assert ns(**bad) == status


def test_nothing_to_do():
    assert ns(count=0, src=None, dst=None, lds=None, ldd=None, ws=None, nws=0) == 0


def test_workspace_bytes():
    n = fs.fsdp_newton_schulz_workspace_bytes
    assert n(0, 8, 8) == 0 and n(1, 0, 8) == 0 and n(1, 1 << 21, 8) == 0
    assert n(1, 100, 300) == n(1, 300, 100) >= 2 * 4 * 100 * 300 + 2 * 4 * 100 * 100
    for side in (64, 300):                                              # in one launch, and with planes
        assert n(1, side, side) < n(2, side, side) <= n(64, side, side) == n(1000, side, side)
    assert n(8, 4096, 11008) == n(1, 4096, 11008) < 1 << 30             # one at a time


LAYOUT = dict(shapes=[(8, 16), (16,), (16, 8), (3, 4, 5), (0, 4), (9, 1), ()], n_ranks=2, mode=fs.FSDP_ZERO1)


def muon(layout=None, **k):
    a = dict(ids=(0, 2, 3), grads=(P, P), gdt=1, master=P, mom=P, params=(P, P), pdt=1, hp=fs.MuonHparams(), coeffs=None, ws=P,
             nws=1 << 30)
    a.update(k)
    L = layout or fs.Layout(**LAYOUT)
    hp = None if a["hp"] is None else C.byref(a["hp"])
    return fs.lib().fsdp_zero1_muon_broadcast(L.handle, len(a["ids"]), arr(C.c_int32, a["ids"]), arr(C.c_void_p, a["grads"]), a["gdt"],
                                              a["master"], a["mom"], arr(C.c_void_p, a["params"]), a["pdt"], hp,
                                              arr(C.c_float, a["coeffs"]), a["ws"], a["nws"], None)


H = fs.MuonHparams


@pytest.mark.parametrize("bad,status", [
    (dict(ids=(0, 0)), EINVAL), (dict(ids=(7,)), EINVAL), (dict(ids=(-1,)), EINVAL), (dict(ids=(1,)), ESHAPE), (dict(ids=(4,)), ESHAPE),
    (dict(ids=(5,)), ESHAPE), (dict(ids=(6,)), ESHAPE), (dict(gdt=2), EDTYPE), (dict(pdt=3), EDTYPE), (dict(master=None), EINVAL),
    (dict(pdt=0), EINVAL), (dict(grads=None), EINVAL), (dict(params=None), EINVAL), (dict(grads=(P, None)), EINVAL),
    (dict(params=(None, P)), EINVAL), (dict(grads=(P, P + 8)), EALIGN), (dict(params=(P + 2, P)), EALIGN), (dict(mom=None), EINVAL),
    (dict(mom=P + 4), EALIGN), (dict(master=P + 4), EALIGN), (dict(hp=None), EINVAL), (dict(hp=H(lr=NAN)), EINVAL),
    (dict(hp=H(lr=-1.0)), EINVAL), (dict(hp=H(momentum=1.0)), EINVAL), (dict(hp=H(momentum=-0.1)), EINVAL),
    (dict(hp=H(weight_decay=-1.0)), EINVAL), (dict(hp=H(weight_decay=INF)), EINVAL), (dict(hp=H(eps=0.0)), EINVAL),
    (dict(hp=H(steps=0)), EINVAL), (dict(hp=H(steps=65)), EINVAL), (dict(hp=H(scale=3)), EINVAL), (dict(hp=H(scale=-1)), EINVAL),
    (dict(hp=H(steps=1), coeffs=(5, 0, 0)), EINVAL), (dict(ws=None), EINVAL), (dict(nws=1000), EINVAL), (dict(ws=P + 8), EALIGN),
])
def test_muon_refused(bad, status):
    assert muon(**bad) == status


def test_muon_wants_a_zero1_layout():
    for mode in (fs.FSDP_FLAT, fs.FSDP_DIM0):
        L = fs.Layout([(8, 16)], n_ranks=2, mode=mode)
        assert muon(L, ids=(0,)) == EINVAL and fs.fsdp_zero1_muon_workspace_bytes(L, [0]) == 0


def test_muon_workspace_bytes():
    L = fs.Layout(**LAYOUT)
    n = fs.fsdp_zero1_muon_workspace_bytes
    assert n(L, []) == 0 and n(L, [1]) == 0 and n(L, [0, 0]) == 0 and n(L, [9]) == 0
    assert 0 < n(L, [0]) < n(L, [0, 2])                      # 8 x 16 and 16 x 8 go together
    assert n(L, [0, 3]) == max(n(L, [0]), n(L, [3]))         # others one after the other
    assert muon(ids=(), ws=None, nws=0) == 0


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fs.fsdp_newton_schulz(x, x)
    with pytest.raises(TypeError, match="unsupported dtype"):
        fs.fsdp_newton_schulz(x.half(), x.half())
    with pytest.raises(ValueError, match="destinations"):
        fs.fsdp_newton_schulz([x, x], [x])
    with pytest.raises(ValueError, match="coeffs"):
        fs._coeffs([(1.0, 2.0)], 1)
    with pytest.raises(ValueError, match="unknown scale"):
        fs.MuonHparams(scale="big")
    L = fs.Layout([(8, 16)], n_ranks=2, mode=fs.FSDP_ZERO1)
    with pytest.raises(ValueError, match="replicas"):
        fs.fsdp_zero1_muon_broadcast(L, [0], [x], x, x, [x, x])
