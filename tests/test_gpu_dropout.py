"""fsdp_dropout against the generator's published round function, bit for bit."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def reference(x, spec, residual):
    """The same fp32 operations on the CPU's rounding rules: multiply, add, round once."""
    keep = lu.keep_mask(*x.shape, spec)
    y = torch.where(keep, x.float() * torch.tensor(1.0 / (1.0 - spec.p), dtype=F32, device=x.device), torch.zeros((), device=x.device))
    if residual is not None:
        y = y + residual.float()
    return y.to(x.dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (1, 4096, 0, 0), (7, 33, 0, 0), (64, 256, 0, 0), (77, 1001, 0, 0),
                                                  (50, 120, 8, 0), (50, 120, 3, 1), (33, 2048, 0, 4), (300, 513, 7, 3),
                                                  (4099, 72, 0, 0)])
def test_dropout_bits(rows, cols, pad, offset, res, dtype):
    g = lu.gen(11)
    ld = cols + pad if pad else None
    x = lu.matrix(rows, cols, dtype, 1.0, g, ld, offset)
    r = lu.matrix(rows, cols, dtype, 1.0, g, ld, offset) if res else None
    for spec in (fs.DropoutSpec(0.1, 42, layer=3), fs.DropoutSpec(0.5, 2 ** 63 + 17, layer=2 ** 32 - 1, row0=2 ** 32 - 5)):
        y, buf = lu.empty_matrix(rows, cols, dtype, ld, offset)
        fs.fsdp_dropout(x, y, spec, residual=r)
        fs.fsdp_check_status()
        assert torch.equal(y, reference(x, spec, r))
        assert lu.untouched(y, buf)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dropout_in_place_and_special_values(dtype):
    x = torch.randn(40, 96, device="cuda").to(dtype)
    x[0] = float("inf")
    x[1] = float("nan")
    spec = fs.DropoutSpec(0.4, 5)
    keep = lu.keep_mask(40, 96, spec)
    y = torch.empty_like(x)
    fs.fsdp_dropout(x, y, spec)
    assert (y[~keep] == 0).all()                       # a dropped infinity or NaN is 0
    assert y[0][keep[0]].isinf().all() and y[1][keep[1]].isnan().all()
    z = x.clone()
    fs.fsdp_dropout(z, z, spec)
    assert torch.equal(z[2:], y[2:])
    r = torch.randn(40, 96, device="cuda").to(dtype)
    want = torch.empty_like(x)
    fs.fsdp_dropout(x, want, spec, residual=r)
    fs.fsdp_dropout(x, r, spec, residual=r)
    assert torch.equal(r[2:], want[2:])


@pytest.mark.parametrize("spec", [None, "p0"])
def test_no_dropout_copies(spec):
    x = torch.randn(33, 70, device="cuda")
    y = torch.empty_like(x)
    fs.fsdp_dropout(x, y, None if spec is None else fs.DropoutSpec(0.0, 1))
    assert torch.equal(x, y)


def test_split_rows_meet_the_same_mask():
    x = torch.randn(100, 50, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    fs.fsdp_dropout(x, a, fs.DropoutSpec(0.2, 9, layer=4))
    for r0, r1 in ((0, 37), (37, 38), (38, 100)):
        fs.fsdp_dropout(x[r0:r1], b[r0:r1], fs.DropoutSpec(0.2, 9, layer=4, row0=r0))
    assert torch.equal(a, b)


def test_empty():
    x = torch.empty(0, 16, device="cuda")
    fs.fsdp_dropout(x, x, fs.DropoutSpec(0.2, 9))
    x = torch.empty(16, 0, device="cuda")
    fs.fsdp_dropout(x, x, fs.DropoutSpec(0.2, 9))
    fs.fsdp_check_status()
