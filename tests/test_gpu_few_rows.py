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
