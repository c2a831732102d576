"""The linear kernels that large fp32 products, slabs and long matrices take, and dropout of
matrices that are not in step."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu
from test_gpu_dropout import reference

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("rows,cin,cout,pad,offset", [(1000, 2048, 2048, 0, 0), (2600, 640, 2500, 0, 0), (1100, 1280, 2405, 0, 1),
                                                      (1300, 2048, 1440, 4, 0), (70, 1100, 900, 3, 0)])
def test_fp32_epilogues_on_the_tensor_cores(rows, cin, cout, pad, offset, act, p):
    """Pairs with 128 and 256 columns, whole and with halved tiles in the last wave, and a split
    size; rows of 32-byte, 16-byte and no alignment, ragged on every side; dgrad at the transposed widths."""
    g = lu.gen(91)
    ld = cout + pad
    x, w = lu.matrix(rows, cin, F32, 1.0, g, None, offset), lu.matrix(cout, cin, F32, 0.02, g, None, offset)
    bias = lu.matrix(1, cout, F32, 0.5, g, None, offset)[0]
    res = lu.matrix(rows, cout, F32, 1.0, g, ld, offset)
    spec = fs.DropoutSpec(p, 5, 6, row0=2 ** 32 - 40) if p else None
    y, ybuf = lu.empty_matrix(rows, cout, F32, ld, offset)
    z, zbuf = lu.empty_matrix(rows, cout, F32, ld, offset)
    ws = lu.workspace(rows, cin, cout, F32)
    fs.fsdp_linear_forward(x, w, y, bias=bias, act=act, preact=z, dropout=spec, residual=res, workspace=ws)
    want, zwant, bound = lu.forward64(x, w, bias, act, spec, res)
    lu.check(z, zwant, bound, "preact")
    lu.check(y, want, 1.13 / (1 - p) * bound + 2.0 ** -20 * (zwant.abs() / (1 - p) + res.double().abs()), "y")
    assert lu.untouched(y, ybuf) and lu.untouched(z, zbuf)
    inplace = res.clone(memory_format=torch.preserve_format) if pad == 0 else res
    fs.fsdp_linear_forward(x, w, inplace, bias=bias, act=act, dropout=spec, residual=inplace, workspace=ws)
    assert torch.equal(inplace, y)
    # dgrad: dz [rows, cin] through a weight [cin, cout] gives dx [rows, cout]
    wt = lu.matrix(cin, cout, F32, 0.02, g, ld, offset)
    dx, xbuf = lu.empty_matrix(rows, cout, F32, ld, offset)
    fs.fsdp_linear_dgrad(x, wt, dx, act=act, preact=z if act != "none" else None, dropout=spec, residual=y,
                         workspace=lu.workspace(rows, cout, cin, F32))
    fs.fsdp_check_status()
    h, M = x.double() @ wt.double(), x.double().abs() @ wt.double().abs()
    want = lu.drop64(h, spec) * lu.act_grad64(z.double(), act) + y.double()
    lu.check(dx, want, 1.13 / (1 - p) * lu.product_bound(cin, M, F32) + 2.0 ** -20 * (2 * h.abs() + y.double().abs()), "dx")
    assert lu.untouched(dx, xbuf)


@pytest.mark.parametrize("grad_dtype", [F32, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cin,cout,offset", [(16384, 128, 128, 0), (20011, 130, 100, 1), (9000, 250, 257, 0)])
def test_wgrad_by_slabs_of_rows(rows, cin, cout, offset, dtype, accumulate, grad_dtype):
    g = lu.gen(92)
    dz, x = lu.matrix(rows, cout, dtype, 1e-3, g, None, offset), lu.matrix(rows, cin, dtype, 1.0, g, None, offset)
    dw, wbuf = lu.empty_matrix(cout, cin, grad_dtype, None, offset)
    db, bbuf = lu.empty_matrix(1, cout, grad_dtype, None, offset)
    dw.fill_(0.25)
    db.fill_(0.25)
    fs.fsdp_linear_wgrad(dz, x, dw, db[0], accumulate=accumulate, workspace=lu.workspace(rows, cin, cout, dtype))
    fs.fsdp_check_status()
    add = 0.25 if accumulate else 0.0
    want_w, want_b = dz.double().t() @ x.double() + add, dz.double().sum(0) + add
    Mw, Mb = dz.double().abs().t() @ x.double().abs(), dz.double().abs().sum(0)
    lu.check(dw, want_w, lu.product_bound(rows, Mw, dtype) + 2.0 ** -23 * want_w.abs(), "dw")
    lu.check(db[0], want_b, (rows / 64 + 64) * 2.0 ** -24 * Mb + 2.0 ** -23 * want_b.abs(), "db")
    assert lu.untouched(dw, wbuf) and lu.untouched(db, bbuf)


def test_gradients_past_32_bits():
    """dgrad with a dx, and wgrad with a dz, of more than 2^31 elements: the last rows and columns."""
    rows, wide, narrow = 70000, 32000, 64
    g = lu.gen(93)
    small, w = lu.matrix(rows, narrow, BF16, 1.0, g), lu.matrix(narrow, wide, BF16, 0.1, g)
    spec = fs.DropoutSpec(0.2, 11, 3)
    dx = torch.empty(rows, wide, dtype=BF16, device="cuda")
    fs.fsdp_linear_dgrad(small, w, dx, dropout=spec)
    tail = small[-300:]
    tailspec = fs.DropoutSpec(0.2, 11, 3, row0=rows - 300)
    h, M = tail.double() @ w.double(), tail.double().abs() @ w.double().abs()
    lu.check(dx[-300:], lu.drop64(h, tailspec), 1.25 * lu.product_bound(narrow, M, BF16) + 2.0 ** -20 * h.abs(), "dx")
    # wgrad of that dx as dz, both ways round: [wide, narrow] and [narrow, wide]
    for dz, x in ((dx, small), (small, dx)):
        dw = torch.empty(dz.shape[1], x.shape[1], device="cuda")
        db = torch.empty(dz.shape[1], device="cuda")
        ws = lu.workspace(rows, x.shape[1], dz.shape[1], BF16)
        fs.fsdp_linear_wgrad(dz, x, dw, db, workspace=ws)
        fs.fsdp_check_status()
        a, b = dz[:, -64:].double(), x[:, -64:].double()
        lu.check(dw[-64:, -64:], a.t() @ b, lu.product_bound(rows, a.abs().t() @ b.abs(), BF16), "dw")
        lu.check(db[-64:], a.sum(0), (rows / 8 + 64) * 2.0 ** -24 * a.abs().sum(0), "db")


# offsets and paddings of x, residual and y; in step only where all agree modulo 16 bytes
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 5), (1, 700), (3, 255), (3, 256), (3, 257), (40, 1001), (129, 64)])
@pytest.mark.parametrize("offsets,pads", [((0, 1, 0), (0, 0, 0)), ((1, 0, 3), (0, 0, 0)), ((0, 0, 0), (8, 0, 1)), ((2, 2, 3), (3, 3, 3)),
                                          ((5, 5, 5), (1, 2, 8)), ((8, 0, 4), (0, 4, 8))])
@pytest.mark.parametrize("res", [False, True])
def test_dropout_of_matrices_out_of_step(rows, cols, offsets, pads, res, dtype):
    g = lu.gen(94)
    x = lu.matrix(rows, cols, dtype, 1.0, g, cols + pads[0], offsets[0])
    r = lu.matrix(rows, cols, dtype, 1.0, g, cols + pads[1], offsets[1]) if res else None
    y, buf = lu.empty_matrix(rows, cols, dtype, cols + pads[2], offsets[2])
    for spec in (fs.DropoutSpec(0.3, 42, layer=3), fs.DropoutSpec(0.5, 2 ** 63 + 17, layer=2 ** 32 - 1, row0=2 ** 32 - 2)):
        fs.fsdp_dropout(x, y, spec, residual=r)
        fs.fsdp_check_status()
        assert torch.equal(y, reference(x, spec, r)) and lu.untouched(y, buf)
    fs.fsdp_dropout(x, y, None, residual=r)
    assert torch.equal(y, x if r is None else (x.float() + r.float()).to(dtype)) and lu.untouched(y, buf)
