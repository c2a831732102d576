"""Linear layers (forward, dgrad, wgrad) against their definitions in 64 bits."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = [BF16, F32]

# rows, in, out: one token to several tiles, K and both tile axes ragged, widths of no
# 16-byte multiple, and sizes at and next to the tile edges
SHAPES = [(1, 32, 32), (1, 2048, 2048), (3, 1, 1), (2, 7, 5), (31, 64, 128), (33, 65, 129), (128, 128, 128), (127, 200, 256),
          (129, 192, 257), (333, 1001, 777), (256, 512, 512), (640, 320, 1000), (1000, 2048, 96), (77, 5504, 256),
          (2048, 256, 512)]


def _tensors(rows, cin, cout, dtype, seed, pad=0, offset=0):
    g = lu.gen(seed)
    ld = (lambda n: n + pad) if pad else (lambda n: None)
    x = lu.matrix(rows, cin, dtype, 1.0, g, ld(cin), offset)
    w = lu.matrix(cout, cin, dtype, 0.02 if cin > 100 else 0.3, g, ld(cin), offset)
    return g, x, w, ld


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_product(shape, dtype):
    rows, cin, cout = shape
    _, x, w, _ = _tensors(rows, cin, cout, dtype, 1)
    y, buf = lu.empty_matrix(rows, cout, dtype)
    fs.fsdp_linear_forward(x, w, y, workspace=lu.workspace(*shape, dtype))
    fs.fsdp_check_status()
    want, _, bound = lu.forward64(x, w, None, "none", None, None)
    lu.check(y, want, bound, "y")
    assert lu.untouched(y, buf)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("shape,pad,offset", [((45, 96, 200), 0, 0), ((130, 72, 264), 8, 0), ((67, 33, 101), 3, 1),
                                              ((300, 128, 128), 0, 5), ((5, 640, 72), 0, 0)])
def test_forward_epilogue(shape, pad, offset, act, dtype):
    rows, cin, cout = shape
    g, x, w, ld = _tensors(rows, cin, cout, dtype, 2, pad, offset)
    bias = lu.matrix(1, cout, dtype, 0.5, g, None, offset)[0]
    residual = lu.matrix(rows, cout, dtype, 1.0, g, ld(cout), offset)
    spec = fs.DropoutSpec(0.3, 0x1234567890ABCDEF, layer=7, row0=5)
    y, ybuf = lu.empty_matrix(rows, cout, dtype, ld(cout), offset)
    z, zbuf = lu.empty_matrix(rows, cout, dtype, ld(cout), offset)
    fs.fsdp_linear_forward(x, w, y, bias=bias, act=act, preact=z, dropout=spec, residual=residual,
                           workspace=lu.workspace(*shape, dtype))
    fs.fsdp_check_status()
    want, zwant, bound = lu.forward64(x, w, bias, act, spec, residual)
    lu.check(z, zwant, bound, "preact")
    # the activations' slopes are below 1.13; the fp32 epilogue's own roundings below 2^-20
    ebound = 1.13 / 0.7 * bound + 2.0 ** -20 * (zwant.abs() / 0.7 + residual.double().abs())
    lu.check(y, want, ebound, "y")
    assert lu.untouched(y, ybuf) and lu.untouched(z, zbuf)
    # residual in place gives the same bits
    r2 = residual.clone() if pad == 0 else residual
    fs.fsdp_linear_forward(x, w, r2, bias=bias, act=act, dropout=spec, residual=r2, workspace=lu.workspace(*shape, dtype))
    assert torch.equal(r2, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_dgrad_product(shape, dtype):
    rows, cin, cout = shape
    g, _, w, _ = _tensors(rows, cin, cout, dtype, 3)
    dz = lu.matrix(rows, cout, dtype, 1e-3, g)
    dx, buf = lu.empty_matrix(rows, cin, dtype)
    fs.fsdp_linear_dgrad(dz, w, dx, workspace=lu.workspace(*shape, dtype))
    fs.fsdp_check_status()
    M = dz.double().abs() @ w.double().abs()
    lu.check(dx, dz.double() @ w.double(), lu.product_bound(cout, M, dtype), "dx")
    assert lu.untouched(dx, buf)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("shape,pad,offset", [((45, 200, 96), 0, 0), ((130, 264, 72), 8, 0), ((67, 101, 33), 3, 1),
                                              ((300, 128, 128), 0, 5), ((5, 72, 640), 0, 0)])
def test_dgrad_epilogue(shape, pad, offset, act, dtype):
    rows, cin, cout = shape
    g, _, w, ld = _tensors(rows, cin, cout, dtype, 4, pad, offset)
    dz = lu.matrix(rows, cout, dtype, 1.0, g, ld(cout), offset)
    z = lu.matrix(rows, cin, dtype, 1.5, g, ld(cin), offset)
    residual = lu.matrix(rows, cin, dtype, 1.0, g, ld(cin), offset)
    spec = fs.DropoutSpec(0.25, 99, layer=1)
    dx, buf = lu.empty_matrix(rows, cin, dtype, ld(cin), offset)
    fs.fsdp_linear_dgrad(dz, w, dx, act=act, preact=z if act != "none" else None, dropout=spec, residual=residual,
                         workspace=lu.workspace(*shape, dtype))
    fs.fsdp_check_status()
    h = dz.double() @ w.double()
    M = dz.double().abs() @ w.double().abs()
    slope = lu.act_grad64(z.double(), act)
    want = lu.drop64(h, spec) * slope + residual.double()
    bound = 1.13 / 0.75 * lu.product_bound(cout, M, dtype) + 2.0 ** -20 * (2 * h.abs() + residual.double().abs())
    lu.check(dx, want, bound, "dx")
    assert lu.untouched(dx, buf)


@pytest.mark.parametrize("dtype,grad_dtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("shape,pad,offset", [((1, 32, 32), 0, 0), ((45, 96, 200), 0, 0), ((130, 264, 72), 8, 0), ((67, 33, 101), 3, 1),
                                              ((300, 128, 128), 0, 5), ((4096, 64, 32), 0, 0), ((1000, 256, 777), 0, 0),
                                              ((2, 1, 1), 0, 0), ((515, 384, 512), 0, 0)])
def test_wgrad(shape, pad, offset, accumulate, dtype, grad_dtype):
    rows, cin, cout = shape
    g = lu.gen(5)
    ld = (lambda n: n + pad) if pad else (lambda n: None)
    dz = lu.matrix(rows, cout, dtype, 1e-3, g, ld(cout), offset)
    x = lu.matrix(rows, cin, dtype, 1.0, g, ld(cin), offset)
    dw, wbuf = lu.empty_matrix(cout, cin, grad_dtype, ld(cin), offset)
    db, bbuf = lu.empty_matrix(1, cout, grad_dtype, None, offset)
    db = db[0]
    want_w, want_b = dz.double().t() @ x.double(), dz.double().sum(0)
    Mw, Mb = dz.double().abs().t() @ x.double().abs(), dz.double().abs().sum(0)
    bw = lu.product_bound(rows, Mw, dtype)
    bb = (rows / 64 + 24) * 2.0 ** -24 * Mb           # at most rows / 64 + 24 fp32 additions in a row
    if accumulate:
        dw.copy_((torch.randn(cout, cin, generator=g, device="cuda") * 1e-2).to(grad_dtype))
        db.copy_((torch.randn(cout, generator=g, device="cuda") * 1e-2).to(grad_dtype))
        want_w, want_b = want_w + dw.double(), want_b + db.double()
        bw, bb = bw + 2.0 ** -23 * want_w.abs(), bb + 2.0 ** -23 * want_b.abs()
    fs.fsdp_linear_wgrad(dz, x, dw, db, accumulate=accumulate, workspace=lu.workspace(*shape, dtype))
    fs.fsdp_check_status()
    lu.check(dw, want_w, bw, "dw")
    lu.check(db, want_b, bb, "db")
    assert lu.untouched(dw, wbuf)
    assert bbuf[:offset].isnan().all() and bbuf[offset + cout:].isnan().all()
