"""The layer operators' argument checks, on the host: every call below carries exactly one
invalid argument, so it is refused before any CUDA call."""
import ctypes as C

import pytest
import torch

import fsdp_sharded_state_gb300 as fs

P = 1 << 20                                     # an aligned address that nothing reads
EINVAL, EDTYPE, ESHAPE, EALIGN, EOVERFLOW = -1, -2, -3, -4, -5


def forward(**k):
    a = dict(rows=4, i=16, o=32, dt=1, x=P, ldx=16, w=P, ldw=16, bias=None, act=0, drop=None, res=None, ldr=0, y=P, ldy=32,
             z=None, ldz=0, ws=None, nws=0)
    a.update(k)
    d = C.byref(a["drop"]) if a["drop"] is not None else None
    return fs.lib().fsdp_linear_forward(a["rows"], a["i"], a["o"], a["dt"], a["x"], a["ldx"], a["w"], a["ldw"], a["bias"],
                                        a["act"], d, a["res"], a["ldr"], a["y"], a["ldy"], a["z"], a["ldz"], a["ws"],
                                        a["nws"], None)


def dgrad(**k):
    a = dict(rows=4, i=16, o=32, dt=1, dz=P, lddz=32, w=P, ldw=16, act=0, z=None, ldz=0, drop=None, res=None, ldr=0, dx=P,
             lddx=16, ws=None, nws=0)
    a.update(k)
    d = C.byref(a["drop"]) if a["drop"] is not None else None
    return fs.lib().fsdp_linear_dgrad(a["rows"], a["i"], a["o"], a["dt"], a["dz"], a["lddz"], a["w"], a["ldw"], a["act"],
                                      a["z"], a["ldz"], d, a["res"], a["ldr"], a["dx"], a["lddx"], a["ws"], a["nws"], None)


def wgrad(**k):
    a = dict(rows=4, i=16, o=32, dt=1, dz=P, lddz=32, x=P, ldx=16, dw=P, lddw=16, db=None, gdt=0, acc=0, ws=None, nws=0)
    a.update(k)
    return fs.lib().fsdp_linear_wgrad(a["rows"], a["i"], a["o"], a["dt"], a["dz"], a["lddz"], a["x"], a["ldx"], a["dw"],
                                      a["lddw"], a["db"], a["gdt"], a["acc"], a["ws"], a["nws"], None)


def dropout(**k):
    a = dict(rows=4, cols=16, dt=1, x=P, ldx=16, drop=None, res=None, ldr=0, y=P, ldy=16)
    a.update(k)
    d = C.byref(a["drop"]) if a["drop"] is not None else None
    return fs.lib().fsdp_dropout(a["rows"], a["cols"], a["dt"], a["x"], a["ldx"], d, a["res"], a["ldr"], a["y"], a["ldy"], None)


@pytest.mark.parametrize("call,bad,status", [
    (forward, dict(dt=2), EDTYPE), (forward, dict(rows=-1), ESHAPE), (forward, dict(i=0), ESHAPE), (forward, dict(o=0), ESHAPE),
    (forward, dict(rows=1 << 31), EOVERFLOW), (forward, dict(act=4), EINVAL), (forward, dict(act=-1), EINVAL),
    (forward, dict(x=None), EINVAL), (forward, dict(w=None), EINVAL), (forward, dict(y=None), EINVAL),
    (forward, dict(x=P + 1), EALIGN), (forward, dict(y=P + 1), EALIGN), (forward, dict(bias=P + 1), EALIGN),
    (forward, dict(dt=0, w=P + 2), EALIGN), (forward, dict(ldx=15), ESHAPE), (forward, dict(ldw=15), ESHAPE),
    (forward, dict(ldy=31), ESHAPE), (forward, dict(res=P, ldr=31), ESHAPE), (forward, dict(z=P, ldz=31), ESHAPE),
    (forward, dict(ldx=1 << 31), EOVERFLOW), (forward, dict(ws=P + 8, nws=1 << 20), EALIGN),
    (forward, dict(drop=fs.DropoutSpec(1.0, 1)), EINVAL), (forward, dict(drop=fs.DropoutSpec(-0.1, 1)), EINVAL),
    (forward, dict(drop=fs.DropoutSpec(float("nan"), 1)), EINVAL), (forward, dict(drop=fs.DropoutSpec(0.1, 1, 0, -1)), EINVAL),
    (forward, dict(drop=fs.DropoutSpec(0.1, 1, 0, (1 << 63) - 2)), EOVERFLOW),
    (forward, dict(dt=0), EINVAL),                            # fp32 operands need the workspace
    (forward, dict(dt=0, ws=P, nws=64), EINVAL),              # and all of it
    (forward, dict(x=P + 2), EINVAL),                         # so do unaligned bf16 ones
    (forward, dict(i=15, ldx=15, ldw=15), EINVAL),
    (dgrad, dict(dt=7), EDTYPE), (dgrad, dict(act=2), EINVAL), (dgrad, dict(act=9), EINVAL), (dgrad, dict(dz=None), EINVAL),
    (dgrad, dict(dx=None), EINVAL), (dgrad, dict(lddz=31), ESHAPE), (dgrad, dict(lddx=15), ESHAPE),
    (dgrad, dict(act=1, z=P, ldz=15), ESHAPE), (dgrad, dict(res=P + 1, ldr=16), EALIGN), (dgrad, dict(ldw=15), ESHAPE),
    (dgrad, dict(drop=fs.DropoutSpec(2.0, 1)), EINVAL), (dgrad, dict(dt=0), EINVAL),
    (wgrad, dict(gdt=2), EDTYPE), (wgrad, dict(dt=-1), EDTYPE), (wgrad, dict(dw=None), EINVAL), (wgrad, dict(dw=P + 2), EALIGN),
    (wgrad, dict(db=P + 2), EALIGN), (wgrad, dict(lddw=15), ESHAPE), (wgrad, dict(ldx=15), ESHAPE), (wgrad, dict(dz=None), EINVAL),
    (wgrad, dict(rows=1 << 40), EOVERFLOW), (wgrad, dict(dt=0), EINVAL), (wgrad, dict(rows=16384), EINVAL),
    (dropout, dict(dt=3), EDTYPE), (dropout, dict(rows=-1), ESHAPE), (dropout, dict(cols=-1), ESHAPE),
    (dropout, dict(x=None), EINVAL), (dropout, dict(y=None), EINVAL), (dropout, dict(y=P + 1), EALIGN),
    (dropout, dict(ldx=15), ESHAPE), (dropout, dict(res=P, ldr=15), ESHAPE),
    (dropout, dict(drop=fs.DropoutSpec(1.5, 1)), EINVAL), (dropout, dict(rows=1 << 30, cols=1 << 11, ldx=1 << 11, ldy=1 << 11), EOVERFLOW),
])
def test_refused(call, bad, status):
    assert call(**bad) == status


def test_nothing_to_do():
    assert forward(rows=0, x=None, y=None) == 0
    assert dgrad(rows=0, dz=None, dx=None) == 0
    assert wgrad(rows=0, dz=None, x=None, acc=1) == 0
    assert dropout(rows=0, x=None, y=None) == 0 and dropout(cols=0, x=None, y=None) == 0


def test_workspace_bytes():
    n = fs.fsdp_linear_workspace_bytes
    assert n(64, 2048, 2048, torch.bfloat16) == 0                       # read where they are
    assert n(64, 2048, 2048, torch.bfloat16, aligned=False) >= 2 * 2048 * (2048 + 64)
    assert n(64, 2047, 2048, torch.bfloat16) == n(64, 2047, 2048, torch.bfloat16, aligned=False) > 0
    assert n(64, 256, 128, torch.float32) >= 3 * 2 * 256 * (128 + 64)   # three bf16 terms of two operands
    assert 0 < n(16384, 64, 32, torch.bfloat16) < 2 << 20               # slabs of a small weight gradient
    assert n(-1, 64, 32, torch.bfloat16) == 0 and n(1, 0, 32, torch.float32) == 0
    for rows, i, o in ((1, 1, 1), (100, 33, 65), (16384, 64, 32), (4096, 5504, 2048)):
        for dt in (torch.bfloat16, torch.float32):
            assert n(rows, i, o, dt, True) <= n(rows, i, o, dt, False)


def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    x, w, y = torch.zeros(4, 16, dtype=bf), torch.zeros(32, 16, dtype=bf), torch.zeros(4, 32, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        fs.fsdp_linear_forward(x, w, y)
    with pytest.raises(TypeError, match="unsupported dtype"):
        fs.fsdp_linear_forward(x.half(), w.half(), y.half())
    with pytest.raises(ValueError, match="matrix"):
        fs.fsdp_linear_forward(x[0], w, y)
    with pytest.raises(ValueError, match="activation"):
        fs._act("swish")
    with pytest.raises(ValueError, match="matrix"):
        fs.fsdp_dropout(x[0], x[0], None)
