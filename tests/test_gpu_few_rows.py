"""fp32 dgrad of one to four rows where the CTAs of a cluster have nothing, or next to nothing, to
add up before they hand their sums on."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
@pytest.mark.parametrize("cin,cout", [(1, 1), (129, 1), (20000, 1), (20001, 3), (4096, 9), (300, 65)])
def test_dgrad_of_few_out_features(rows, cin, cout):
    """One to 65 out-features over 64 warps; many clusters, again and again on a busy stream."""
    g = lu.gen(61)
    dz, w = lu.matrix(rows, cout, F32, 1.0, g), lu.matrix(cout, cin, F32, 1.0, g)
    ws = lu.workspace(rows, cin, cout, F32)
    want, M = dz.double() @ w.double(), dz.double().abs() @ w.double().abs()
    outs = [lu.empty_matrix(rows, cin, F32) for _ in range(20)]
    for dx, _ in outs:
        fs.fsdp_linear_dgrad(dz, w, dx, workspace=ws)
    fs.fsdp_check_status()
    # a sum is at most 2 fused products in a row and the joins of 8 warps and 8 CTAs, 2^-24 each
    for dx, buf in outs:
        lu.check(dx, want, 20 * 2.0 ** -24 * M, "dx")
        assert torch.equal(dx, outs[0][0]) and lu.untouched(dx, buf)


@pytest.mark.parametrize("rows", [1, 4, 5, 16])
def test_forward_needs_no_room_for_the_weight(rows):
    """Up to 16 fp32 rows the weight is read where it is: forward with room for the rows alone;
    dgrad too up to four."""
    g = lu.gen(62)
    cin, cout = 4096, 1100
    x, w, dz = (lu.matrix(r, c, F32, s, g) for r, c, s in ((rows, cin, 1.0), (cout, cin, 0.02), (rows, cout, 1.0)))
    ws = torch.empty(6 * rows * cin + 256, dtype=torch.uint8, device="cuda")
    y, buf = lu.empty_matrix(rows, cout, F32)
    fs.fsdp_linear_forward(x, w, y, workspace=ws)
    want, _, bound = lu.forward64(x, w, None, "none", None, None)
    lu.check(y, want, bound, "y")
    assert lu.untouched(y, buf)
    if rows <= 4:
        dx, buf = lu.empty_matrix(rows, cin, F32)
        fs.fsdp_linear_dgrad(dz, w, dx, workspace=ws)
        lu.check(dx, dz.double() @ w.double(), lu.product_bound(cout, dz.double().abs() @ w.double().abs(), F32), "dx")
        assert lu.untouched(dx, buf)
    fs.fsdp_check_status()


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 17])
@pytest.mark.parametrize("dtype", [torch.bfloat16, F32])
def test_the_counted_workspace_is_enough(rows, dtype):
    """All three calls with exactly the bytes that are asked for, at operands that are not aligned."""
    g = lu.gen(63)
    cin, cout = 1027, 2051
    x, w, dz = (lu.matrix(r, c, dtype, s, g, None, 1) for r, c, s in ((rows, cin, 1.0), (cout, cin, 0.05), (rows, cout, 1.0)))
    n = fs.fsdp_linear_workspace_bytes(rows, cin, cout, dtype, False)
    buf = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[:n]
    y, dx, dw = (torch.empty(r, c, dtype=dtype, device="cuda") for r, c in ((rows, cout), (rows, cin), (cout, cin)))
    fs.fsdp_linear_forward(x, w, y, workspace=ws)
    fs.fsdp_linear_dgrad(dz, w, dx, workspace=ws)
    fs.fsdp_linear_wgrad(dz, x, dw, workspace=ws)
    fs.fsdp_check_status()
    a, b, c = x.double(), w.double(), dz.double()
    for got, l, r, K in ((y, a, b.t(), cin), (dx, c, b, cout), (dw, c.t(), a, rows)):
        lu.check(got, l @ r, lu.product_bound(K, l.abs() @ r.abs(), dtype), "product")
    assert (buf[n:] == 0xA5).all()
