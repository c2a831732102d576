"""Sums of the linear layers' products where the order and the rounding of the additions show."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cin,cout,offset", [(2048, 2048, 0), (2560, 2048, 0), (1000, 1300, 0), (512, 384, 3), (128, 128, 0), (64, 32, 0)])
def test_accumulator_far_above_its_addends(cin, cout, offset, dtype):
    """What is added to an accumulator is rounded to it once: 16384 rows that each add 2^-35 to 1.
    Every partial sum of the addends is a multiple of 2^-35 up to 2^-21, so exact in 32 bits, and
    so is 1 + 2^-21; parts of 4096 rows or fewer, added to 1 by themselves, would leave it as it was
    or round.  For db 2^-20 a row and 2^14, whose sum is exact too."""
    rows = 16384
    dz = torch.full((rows, cout), 2.0 ** -20, dtype=dtype, device="cuda")
    x = torch.full((rows, cin), 2.0 ** -15, dtype=dtype, device="cuda")
    dw, wbuf = lu.empty_matrix(cout, cin, F32, None, offset)
    db, bbuf = lu.empty_matrix(1, cout, F32, None, offset)
    dw.fill_(1.0)
    db.fill_(2.0 ** 14)
    fs.fsdp_linear_wgrad(dz, x, dw, db[0], accumulate=True, workspace=lu.workspace(rows, cin, cout, dtype))
    fs.fsdp_check_status()
    assert (dw == 1 + 2.0 ** -21).all()
    assert (db == 2.0 ** 14 + 2.0 ** -6).all()
    assert lu.untouched(dw, wbuf) and lu.untouched(db, bbuf)
