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


def test_binding_refuses_wrong_tensors():
    x, w, y = (torch.zeros(s, dtype=BF16, device="cuda") for s in ((4, 16), (32, 16), (4, 32)))
    with pytest.raises(TypeError, match="w is"):
        fs.fsdp_linear_forward(x, w.float(), y)
    with pytest.raises(ValueError, match="w is"):
        fs.fsdp_linear_forward(x, torch.zeros(32, 17, dtype=BF16, device="cuda"), y)
    with pytest.raises(ValueError, match="y is"):
        fs.fsdp_linear_forward(x, w, y[:3])
    with pytest.raises(ValueError, match="contiguous"):
        fs.fsdp_linear_forward(torch.zeros(16, 4, dtype=BF16, device="cuda").t(), w, y)
    with pytest.raises(ValueError, match="bias is"):
        fs.fsdp_linear_forward(x, w, y, bias=torch.zeros(31, dtype=BF16, device="cuda"))
    with pytest.raises(fs.FsdpError, match="FSDP_EINVAL"):          # dgrad through an activation needs preact
        fs.fsdp_linear_dgrad(y, w, x, act="gelu")
    with pytest.raises(fs.FsdpError, match="FSDP_EINVAL"):          # fp32 operands need the workspace
        fs.fsdp_linear_forward(x.float(), w.float(), y.float())


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows(dtype):
    x, w = torch.zeros(0, 24, dtype=dtype, device="cuda"), torch.ones(40, 24, dtype=dtype, device="cuda")
    y = torch.zeros(0, 40, dtype=dtype, device="cuda")
    fs.fsdp_linear_forward(x, w, y)
    fs.fsdp_linear_dgrad(y, w, x)
    dw, buf = lu.empty_matrix(40, 24, dtype, 32)
    db = torch.ones(40, dtype=dtype, device="cuda")
    dw.fill_(1)
    fs.fsdp_linear_wgrad(y, x, dw, db, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    fs.fsdp_linear_wgrad(y, x, dw, db)
    fs.fsdp_check_status()
    assert (dw == 0).all() and (db == 0).all() and lu.untouched(dw, buf)


def test_special_values_stay_in_their_rows():
    """An infinity or NaN in a row of x meets that row of y alone; a dropped one becomes 0."""
    x = torch.randn(64, 96, device="cuda").to(BF16)
    w = torch.randn(80, 96, device="cuda").to(BF16)
    spec = fs.DropoutSpec(0.3, 8)
    clean = torch.empty(64, 80, dtype=BF16, device="cuda")
    fs.fsdp_linear_forward(x, w, clean, dropout=spec)
    x[5, 7], x[40, 3] = float("inf"), float("nan")
    y = torch.empty_like(clean)
    fs.fsdp_linear_forward(x, w, y, dropout=spec)
    keep = lu.keep_mask(64, 80, spec)
    rows = [r for r in range(64) if r not in (5, 40)]
    assert torch.equal(y[rows], clean[rows])
    assert (y[~keep] == 0).all()
    assert y[5][keep[5]].isinf().all() and y[40][keep[40]].isnan().all()
    assert torch.equal(y[5][keep[5]] > 0, (w[:, 7] > 0)[keep[5]])


def test_same_bits_every_run_on_any_stream_and_under_capture():
    g = lu.gen(9)
    dz = lu.matrix(3000, 200, BF16, 1.0, g)
    x = lu.matrix(3000, 120, BF16, 1.0, g)
    ws = lu.workspace(3000, 120, 200, BF16)
    outs = [(torch.empty(200, 120, device="cuda"), torch.empty(200, device="cuda")) for _ in range(3)]
    fs.fsdp_linear_wgrad(dz, x, *outs[0], workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fs.fsdp_linear_wgrad(dz, x, *outs[1], workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fsdp_linear_wgrad(dz, x, *outs[2], workspace=ws)
    graph.replay()
    fs.fsdp_check_status()
    for dw, db in outs[1:]:
        assert torch.equal(dw, outs[0][0]) and torch.equal(db, outs[0][1])


@pytest.mark.parametrize("rows", [1, 7, 300, 2000])
def test_forward_rows_do_not_depend_on_the_batch(rows):
    """A row's dropout and residual are its own: rows of a large batch against the same rows
    alone, at the row index that row0 gives (the products' sums may be grouped differently)."""
    g = lu.gen(12)
    x, w = lu.matrix(2000, 256, BF16, 1.0, g), lu.matrix(320, 256, BF16, 0.05, g)
    res = lu.matrix(2000, 320, BF16, 1.0, g)
    y, part = torch.empty(2000, 320, dtype=BF16, device="cuda"), torch.empty(rows, 320, dtype=BF16, device="cuda")
    fs.fsdp_linear_forward(x, w, y, dropout=fs.DropoutSpec(0.5, 3, 1), residual=res)
    r0 = 2000 - rows
    fs.fsdp_linear_forward(x[r0:], w, part, dropout=fs.DropoutSpec(0.5, 3, 1, row0=r0), residual=res[r0:])
    assert (y[r0:].float() - part.float()).abs().max() <= 2.0 ** -6 * y.float().abs().max()
    assert torch.equal(y[r0:] == res[r0:], part == res[r0:])          # the same elements dropped


def test_large_row_index_of_the_mask():
    """row0 near 2^32: rows on both sides of the counter's word boundary, fused and alone."""
    g = lu.gen(13)
    x, w = lu.matrix(600, 64, BF16, 1.0, g), lu.matrix(512, 64, BF16, 0.3, g)
    spec = fs.DropoutSpec(0.5, 77, 2, row0=2 ** 32 - 290)
    y = torch.empty(600, 512, dtype=BF16, device="cuda")
    fs.fsdp_linear_forward(x, w, y, dropout=spec)
    plain = torch.empty_like(y)
    fs.fsdp_linear_forward(x, w, plain)
    keep = lu.keep_mask(600, 512, spec)
    assert torch.equal(y != 0, keep & (plain != 0))
    alone = torch.empty_like(y)
    fs.fsdp_dropout(plain, alone, spec)
    assert torch.equal(alone != 0, keep & (plain != 0))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("rows,cin,cout,pad", [(1300, 2048, 1408, 0), (1300, 2048, 1400, 0), (1100, 2048, 1405, 0), (1030, 2048, 1440, 8)])
def test_pair_kernels_epilogues(rows, cin, cout, pad, act, p):
    """Sizes with enough tiles for the CTA pairs: rows of 32-byte, 16-byte and no alignment,
    ragged on every side; forward, then dgrad at the transposed widths."""
    g = lu.gen(21)
    x = lu.matrix(rows, cin, BF16, 1.0, g)
    w = lu.matrix(cout, cin, BF16, 0.02, g)
    bias = lu.matrix(1, cout, BF16, 0.5, g)[0]
    ld = cout + pad
    res = lu.matrix(rows, cout, BF16, 1.0, g, ld)
    spec = fs.DropoutSpec(p, 5, 6, row0=3) if p else None
    y, ybuf = lu.empty_matrix(rows, cout, BF16, ld)
    z, zbuf = lu.empty_matrix(rows, cout, BF16, ld)
    fs.fsdp_linear_forward(x, w, y, bias=bias, act=act, preact=z, dropout=spec, residual=res,
                           workspace=lu.workspace(rows, cin, cout, BF16))
    want, zwant, bound = lu.forward64(x, w, bias, act, spec, res)
    lu.check(z, zwant, bound, "preact")
    lu.check(y, want, 1.13 / (1 - p) * bound + 2.0 ** -20 * (zwant.abs() / (1 - p) + res.double().abs()), "y")
    assert lu.untouched(y, ybuf) and lu.untouched(z, zbuf)
    # dgrad: dz [rows, cin] through a weight [cin, cout] gives dx [rows, cout]
    wt = lu.matrix(cin, cout, BF16, 0.02, g)
    dx, xbuf = lu.empty_matrix(rows, cout, BF16, ld)
    fs.fsdp_linear_dgrad(x, wt, dx, act=act, preact=z if act != "none" else None, dropout=spec, residual=res,
                         workspace=lu.workspace(rows, cout, cin, BF16))
    fs.fsdp_check_status()
    h = x.double() @ wt.double()
    M = x.double().abs() @ wt.double().abs()
    want = lu.drop64(h, spec) * lu.act_grad64(z.double(), act) + res.double()
    lu.check(dx, want, 1.13 / (1 - p) * lu.product_bound(cin, M, BF16) + 2.0 ** -20 * (2 * h.abs() + res.double().abs()), "dx")
    assert lu.untouched(dx, xbuf)


@pytest.mark.parametrize("dtype,grad_dtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,cin,cout", [(1500, 1408, 1300), (777, 2100, 1001), (9000, 40, 130), (20000, 8, 3)])
def test_wgrad_pairs_and_slabs(rows, cin, cout, accumulate, dtype, grad_dtype):
    g = lu.gen(22)
    dz, x = lu.matrix(rows, cout, dtype, 1e-3, g), lu.matrix(rows, cin, dtype, 1.0, g)
    dw = torch.full((cout, cin), 0.25, dtype=grad_dtype, device="cuda")
    db = torch.full((cout,), 0.25, dtype=grad_dtype, device="cuda")
    fs.fsdp_linear_wgrad(dz, x, dw, db, accumulate=accumulate, workspace=lu.workspace(rows, cin, cout, dtype))
    fs.fsdp_check_status()
    add = 0.25 if accumulate else 0.0
    want_w, want_b = dz.double().t() @ x.double() + add, dz.double().sum(0) + add
    Mw, Mb = dz.double().abs().t() @ x.double().abs(), dz.double().abs().sum(0)
    lu.check(dw, want_w, lu.product_bound(rows, Mw, dtype) + 2.0 ** -23 * want_w.abs(), "dw")
    lu.check(db, want_b, (rows / 64 + 64) * 2.0 ** -24 * Mb + 2.0 ** -23 * want_b.abs(), "db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 13, 16, 17])
@pytest.mark.parametrize("cin,cout,offset", [(300, 520, 0), (2048, 136, 0), (129, 77, 1), (1, 3, 0)])
def test_few_rows(rows, cin, cout, offset, dtype):
    g = lu.gen(31)
    x, w = lu.matrix(rows, cin, dtype, 1.0, g, None, offset), lu.matrix(cout, cin, dtype, 0.05, g, None, offset)
    bias = lu.matrix(1, cout, dtype, 0.5, g, None, offset)[0]
    res = lu.matrix(rows, cout, dtype, 1.0, g)
    spec = fs.DropoutSpec(0.4, 2 ** 40 + 3, 5, row0=2 ** 32 - 2)
    y, ybuf = lu.empty_matrix(rows, cout, dtype, None, offset)
    z, zbuf = lu.empty_matrix(rows, cout, dtype, None, offset)
    ws = lu.workspace(rows, cin, cout, dtype)
    fs.fsdp_linear_forward(x, w, y, bias=bias, act="gelu", preact=z, dropout=spec, residual=res, workspace=ws)
    fs.fsdp_check_status()
    want, zwant, bound = lu.forward64(x, w, bias, "gelu", spec, res)
    lu.check(z, zwant, bound, "preact")
    lu.check(y, want, 1.13 / 0.6 * bound + 2.0 ** -20 * (zwant.abs() / 0.6 + res.double().abs()), "y")
    assert lu.untouched(y, ybuf) and lu.untouched(z, zbuf)
    # dgrad at the same sizes: dz = res [rows, cout] through w, with x as the pre-activation
    dx, xbuf = lu.empty_matrix(rows, cin, dtype, None, offset)
    fs.fsdp_linear_dgrad(res, w, dx, act="silu", preact=x, dropout=spec, workspace=ws)
    fs.fsdp_check_status()
    h, M = res.double() @ w.double(), res.double().abs() @ w.double().abs()
    want = lu.drop64(h, spec) * lu.act_grad64(x.double(), "silu")
    lu.check(dx, want, 1.13 / 0.6 * lu.product_bound(cout, M, dtype) + 2.0 ** -20 * 2 * h.abs(), "dx")
    assert lu.untouched(dx, xbuf)


def test_offsets_past_32_bits():
    """Outputs of more than 2^31 elements: the last rows against the same rows computed alone."""
    rows, cin, cout = 70000, 64, 32000
    g = lu.gen(41)
    x, w = lu.matrix(rows, cin, BF16, 1.0, g), lu.matrix(cout, cin, BF16, 0.1, g)
    spec = fs.DropoutSpec(0.2, 11, 3)
    y = torch.empty(rows, cout, dtype=BF16, device="cuda")
    fs.fsdp_linear_forward(x, w, y, act="gelu", dropout=spec)
    part = torch.empty(300, cout, dtype=BF16, device="cuda")
    fs.fsdp_linear_forward(x[-300:], w, part, act="gelu", dropout=fs.DropoutSpec(0.2, 11, 3, row0=rows - 300))
    fs.fsdp_check_status()
    assert torch.equal(y[-300:] == 0, part == 0)
    assert (y[-300:].float() - part.float()).abs().max() <= 2.0 ** -6 * part.float().abs().max()
    z = torch.empty_like(y)
    fs.fsdp_dropout(y, z, spec)
    small = torch.empty_like(part)
    fs.fsdp_dropout(y[-300:], small, fs.DropoutSpec(0.2, 11, 3, row0=rows - 300))
    fs.fsdp_check_status()
    assert torch.equal(z[-300:], small)


@pytest.mark.parametrize("dtype", DTYPES)
def test_views_of_wide_buffers(dtype):
    """Operands and results as column ranges of wider matrices, weights as a view of a flat
    buffer at an odd element."""
    g = lu.gen(42)
    big = lu.matrix(900, 1500, dtype, 1.0, g)
    x, res = big[:, 100:612], big[:, 700:1100]
    flat = lu.matrix(1, 400 * 512 + 3, dtype, 0.05, g)[0]
    w = flat[3:].view(400, 512)
    out = torch.full((900, 1000), 7.0, dtype=dtype, device="cuda")
    y = out[:, 333:733]
    fs.fsdp_linear_forward(x, w, y, residual=res, workspace=lu.workspace(900, 512, 400, dtype))
    fs.fsdp_check_status()
    want, z, bound = lu.forward64(x, w, None, "none", None, res)
    lu.check(y, want, bound + 2.0 ** -20 * (z.abs() + res.double().abs()), "y")
    assert (out[:, :333] == 7).all() and (out[:, 733:] == 7).all()


@pytest.mark.parametrize("dtype,ld", [(BF16, 8), (BF16, 1), (F32, 4), (F32, 1)])
@pytest.mark.parametrize("rows,cin,cout", [(1000, 200, 9001), (1031, 500, 9001), (1031, 1100, 4333), (1500, 2300, 2051), (63, 2300, 4333)])
def test_bias_gradient_of_wide_layers(rows, cin, cout, dtype, ld):
    # one, two, five and nine tiles to a row of tiles share dz's columns out; rows that start at
    # multiples of 16 bytes (the rest of the stride is NaN) and anywhere, the last row's end is
    # the buffer's.  A lane adds at most every second row, four at a time.
    g = lu.gen(31)
    dz = lu.matrix(rows, cout, dtype, 1e-3, g, (cout + ld - 1) // ld * ld)
    x = lu.matrix(rows, cin, dtype, 1.0, g)
    dw, db = torch.empty(cout, cin, dtype=F32, device="cuda"), torch.empty(cout, dtype=F32, device="cuda")
    fs.fsdp_linear_wgrad(dz, x, dw, db, workspace=lu.workspace(rows, cin, cout, dtype))
    fs.fsdp_check_status()
    lu.check(db, dz.double().sum(0), (rows / 8 + 16) * 2.0 ** -24 * dz.double().abs().sum(0), "db")
    M = dz.double().abs().t() @ x.double().abs()
    lu.check(dw, dz.double().t() @ x.double(), lu.product_bound(rows, M, dtype), "dw")


@pytest.mark.parametrize("rows,cin,cout,pad,offset", [(33, 1, 1, 0, 0), (17, 64, 65, 3, 1), (100, 512, 31, 4, 0), (300, 65, 300, 0, 3),
                                                      (2000, 32, 96, 0, 0), (5000, 40, 33, 1, 2)])
@pytest.mark.parametrize("act,p", [("none", 0.0), ("gelu", 0.25)])
def test_small_fp32_products(rows, cin, cout, pad, offset, act, p):
    # on the FMA units: K of one, a step and a bit; the steps' and tiles' ragged ends lie against
    # NaN.  A sum is at most 104 fused products in a row and the joins of 8 warps and 152 slabs
    # (each 2^-24), which the bound of the split products, 104 * 2^-22, covers.
    g = lu.gen(41)
    ld = lambda n: n + pad if pad else None
    x, w = lu.matrix(rows, cin, F32, 1.0, g, ld(cin), offset), lu.matrix(cout, cin, F32, 0.1, g, ld(cin), offset)
    dz, res = lu.matrix(rows, cout, F32, 1e-2, g, ld(cout), offset), lu.matrix(rows, cin, F32, 1.0, g, ld(cin), offset)
    pre = lu.matrix(rows, cin, F32, 1.0, g, ld(cin), offset)
    bias = lu.matrix(1, cout, F32, 1.0, g)[0]
    spec = fs.DropoutSpec(p, 9, 2, 3) if p else None
    ws = lu.workspace(rows, cin, cout, F32)
    y, ybuf = lu.empty_matrix(rows, cout, F32, ld(cout), offset)
    fs.fsdp_linear_forward(x, w, y, bias=bias, act=act, dropout=spec, residual=dz, workspace=ws)
    dx, xbuf = lu.empty_matrix(rows, cin, F32, ld(cin), offset)
    fs.fsdp_linear_dgrad(dz, w, dx, act=act, preact=pre, dropout=spec, residual=res, workspace=ws)
    dw, wbuf = lu.empty_matrix(cout, cin, F32, ld(cin), offset)
    db, bbuf = lu.empty_matrix(1, cout, F32, None, offset)
    fs.fsdp_linear_wgrad(dz, x, dw, db[0], workspace=ws)
    fs.fsdp_check_status()
    want, _, bound = lu.forward64(x, w, bias, act, spec, dz)
    lu.check(y, want, 1.13 / (1 - p) * bound + 2.0 ** -20 * (2 * want.abs() + dz.double().abs()), "y")
    h, M = dz.double() @ w.double(), dz.double().abs() @ w.double().abs()
    want = lu.drop64(h, spec) * lu.act_grad64(pre.double(), act) + res.double()
    lu.check(dx, want, 1.13 / (1 - p) * lu.product_bound(cout, M, F32) + 2.0 ** -20 * (2 * h.abs() + res.double().abs()), "dx")
    M = dz.double().abs().t() @ x.double().abs()
    lu.check(dw, dz.double().t() @ x.double(), lu.product_bound(rows, M, F32), "dw")
    lu.check(db[0], dz.double().sum(0), (rows / 64 + 192) * 2.0 ** -24 * dz.double().abs().sum(0), "db")
    for v, b in ((y, ybuf), (dx, xbuf), (dw, wbuf), (db, bbuf)):
        assert lu.untouched(v, b)
