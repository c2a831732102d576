"""Layer norm's argument checks, on the host: every call below carries exactly one invalid
argument, so it is refused before any CUDA call."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

P = 1 << 20                                     # an aligned address that nothing reads
EINVAL, EDTYPE, ESHAPE, EALIGN, EOVERFLOW = -1, -2, -3, -4, -5
NAN, INF = float("nan"), float("inf")


def forward(**k):
    a = dict(rows=4, cols=16, dt=1, x=P, ldx=16, w=P, b=P, eps=1e-5, y=P, ldy=16, mean=P, rstd=P)
    a.update(k)
    return fs.lib().fsdp_layernorm_forward(a["rows"], a["cols"], a["dt"], a["x"], a["ldx"], a["w"], a["b"], a["eps"], a["y"], a["ldy"],
                                           a["mean"], a["rstd"], None)


def backward(**k):
    a = dict(rows=4, cols=16, dt=1, dy=P, lddy=16, x=P, ldx=16, mean=P, rstd=P, w=P, res=None, ldr=0, dx=P, lddx=16, dw=P, db=P,
             gdt=0, acc=0, ws=P, nws=1 << 20)
    a.update(k)
    return fs.lib().fsdp_layernorm_backward(a["rows"], a["cols"], a["dt"], a["dy"], a["lddy"], a["x"], a["ldx"], a["mean"], a["rstd"],
                                            a["w"], a["res"], a["ldr"], a["dx"], a["lddx"], a["dw"], a["db"], a["gdt"], a["acc"],
                                            a["ws"], a["nws"], None)


@pytest.mark.parametrize("call,bad,status", [
    (forward, dict(dt=2), EDTYPE), (forward, dict(rows=-1), ESHAPE), (forward, dict(cols=0), ESHAPE), (forward, dict(rows=1 << 31), EOVERFLOW),
    (forward, dict(cols=65537, ldx=65537, ldy=65537), EOVERFLOW), (forward, dict(x=None), EINVAL), (forward, dict(y=None), EINVAL),
    (forward, dict(x=P + 1), EALIGN), (forward, dict(y=P + 1), EALIGN), (forward, dict(w=P + 1), EALIGN), (forward, dict(b=P + 1), EALIGN),
    (forward, dict(dt=0, x=P + 2), EALIGN), (forward, dict(mean=P + 2), EALIGN), (forward, dict(rstd=P + 2), EALIGN),
    (forward, dict(ldx=15), ESHAPE), (forward, dict(ldy=15), ESHAPE), (forward, dict(ldx=1 << 31), EOVERFLOW),
    (forward, dict(eps=0.0), EINVAL), (forward, dict(eps=-1e-5), EINVAL), (forward, dict(eps=NAN), EINVAL), (forward, dict(eps=INF), EINVAL),
    (backward, dict(dt=-1), EDTYPE), (backward, dict(gdt=2), EDTYPE), (backward, dict(rows=-1), ESHAPE), (backward, dict(cols=0), ESHAPE),
    (backward, dict(dy=None), EINVAL), (backward, dict(x=None), EINVAL), (backward, dict(dx=None), EINVAL),
    (backward, dict(mean=None), EINVAL), (backward, dict(rstd=None), EINVAL), (backward, dict(mean=P + 2), EALIGN),
    (backward, dict(lddy=15), ESHAPE), (backward, dict(ldx=15), ESHAPE), (backward, dict(lddx=15), ESHAPE),
    (backward, dict(res=P, ldr=15), ESHAPE), (backward, dict(res=P + 1, ldr=16), EALIGN), (backward, dict(w=P + 1), EALIGN),
    (backward, dict(dw=P + 2), EALIGN), (backward, dict(gdt=1, db=P + 1), EALIGN), (backward, dict(ws=None, nws=0), EINVAL),
    (backward, dict(ws=P + 8), EALIGN), (backward, dict(nws=64), EINVAL),
    (backward, dict(rows=(1 << 30), cols=2048, ldx=2048, lddy=2048, lddx=2048), EOVERFLOW),
])
def test_refused(call, bad, status):
    assert call(**bad) == status


def test_nothing_to_do():
    assert forward(rows=0, x=None, y=None) == 0
    assert backward(rows=0, dy=None, x=None, dx=None, mean=None, rstd=None, acc=1, ws=None, nws=0) == 0


def test_workspace_bytes():
    n = fs.fsdp_layernorm_workspace_bytes
    assert n(0, 64) == 0 and n(-1, 64) == 0 and n(4, 0) == 0 and n(4, 65537) == 0
    assert n(1, 1) == 2 * 8 * 4 and n(1, 64) == 2 * 64 * 4
    for cols in (32, 1001, 2048, 4096, 8192, 65536):
        assert 0 < n(1, cols) <= n(1000, cols) <= n(1 << 20, cols) <= 32 * 152 * (cols + 8)


def test_binding_refuses_wrong_tensors():
    bf = torch.bfloat16
    x, v, s = torch.zeros(4, 16, dtype=bf), torch.zeros(16, dtype=bf), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        fs.fsdp_layernorm_forward(x, x)
    with pytest.raises(TypeError, match="unsupported dtype"):
        fs.fsdp_layernorm_forward(x.half(), x.half())
    with pytest.raises(ValueError, match="matrix"):
        fs.fsdp_layernorm_forward(v, v)
    with pytest.raises(ValueError, match="CUDA"):
        fs.fsdp_layernorm_backward(x, x, s, s, x)
