"""Layer norm, forward and backward, against its definition in 64 bits.

The bounds follow from how a result is formed.  A sum over a row of n values passes through at
most D = 32 + 5 + 36 fp32 additions (a thread's 32 elements, a warp's lanes, the warps of a
row), each off by at most 2^-24 of the magnitudes added so far: D 2^-24 times the sum of the
magnitudes.  Differences, products, divisions and square roots round once each.  A sum over T
rows passes through at most T / 100 + 100 additions.  An output is rounded once to its type."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
D = 32 + 5 + 36
EPS = 1e-5

# rows, cols, pad, offset: every way a row is spread over threads, its edges, rows of no
# 16-byte multiple, rows with padding, rows that start at an odd element
SHAPES = [(1, 1, 0, 0), (5, 7, 0, 0), (300, 32, 0, 0), (129, 33, 0, 0), (70, 64, 0, 0), (1, 128, 0, 0), (333, 200, 0, 0), (67, 256, 8, 0),
          (64, 257, 0, 0), (31, 512, 0, 0), (9, 1000, 0, 0), (333, 1001, 0, 0), (40, 1024, 0, 0), (3, 1025, 0, 0), (1, 2048, 0, 0),
          (700, 2048, 0, 0), (5, 2052, 4, 0), (333, 4096, 0, 0), (17, 4100, 0, 3), (12, 8192, 0, 0), (11, 8191, 2, 0), (7, 8200, 0, 0),
          (160, 16384, 0, 0), (3, 20001, 0, 1), (2, 65536, 0, 0), (4, 40000, 0, 0), (65, 96, 3, 1), (20, 1500, 1, 1),
          (5000, 256, 0, 0), (4001, 40, 0, 0), (2500, 2048, 8, 0),
          (9000, 3, 0, 0), (6001, 100, 4, 0), (3001, 500, 0, 1), (900, 5000, 0, 0), (450, 6145, 0, 0), (200, 12000, 8, 0), (150, 33000, 0, 0),
          (16001, 255, 0, 0), (5003, 31, 0, 0), (4000, 509, 0, 1), (3001, 1023, 2, 5), (1500, 2043, 0, 0), (900, 4093, 0, 3), (500, 6143, 0, 0),
          (400, 8189, 0, 2), (300, 16381, 0, 7), (120, 65535, 0, 0), (3, 65536, 3, 1),
          (9001, 200, 0, 0), (3001, 48, 16, 8), (2003, 768, 0, 0), (901, 1536, 8, 0), (700, 2560, 0, 0), (401, 5120, 0, 0), (201, 11008, 0, 8),
          (90, 20480, 0, 0), (40, 49160, 8, 0)]


def _inputs(rows, cols, pad, offset, dtype, seed, mean=0.7, std=1.5):
    g = lu.gen(seed)
    ld = cols + pad
    x = lu.matrix(rows, cols, dtype, std, g, ld, offset)
    x.copy_((x.float() + mean).to(dtype))
    w = lu.matrix(1, cols, dtype, 0.5, g, None, offset)[0]
    w.copy_((w.float() + 1.0).to(dtype))
    b = lu.matrix(1, cols, dtype, 0.5, g, None, offset)[0]
    return g, ld, x, w, b


def forward64(x, w, b):
    """(y, mean, rstd) and the bounds of their errors before the rounding to their types."""
    x, n = x.double(), x.shape[1]
    w = torch.ones(n, device="cuda").double() if w is None else w.double()
    b = torch.zeros(n, device="cuda").double() if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + EPS) ** -0.5
    first = (D + 2) * U * x.abs().mean(1, keepdim=True)            # of the mean that is subtracted
    spread = d.abs().mean(1, keepdim=True) + first                 # magnitudes of the differences
    # what is left of it where it is not taken out: 2^-23 of the root mean square, and a bit
    bmean = (D + 4) * U * spread + 2 * U * mean.abs() + 2.1 * U * var.sqrt()
    brel = 0.5 * (D + 8) * U * (var + first.square()) / (var + EPS) + 4 * U
    yhat = d * rstd
    bd = U * (2 * (d.abs() + first)) + (D + 3) * U * spread + 2.1 * U * var.sqrt()
    by = w.abs() * rstd * bd + (yhat * w).abs() * (brel + 4 * U) + U * b.abs() + 2 * U * (yhat * w + b).abs()
    return (yhat * w + b, by), (mean[:, 0], bmean[:, 0]), (rstd[:, 0], (rstd * brel)[:, 0])


def backward64(dy, x, mean, rstd, w, residual):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    T, n = x.shape
    w = torch.ones(n, device="cuda").double() if w is None else w.double()
    h, g = (x - mean) * rstd, dy * w
    c0, c1 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    m0, m1 = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    dx = rstd * (g - c0 - h * c1)
    bx = rstd * U * (5 * g.abs() + (D + 6) * m0 + (D + 12) * h.abs() * m1)
    if residual is not None:
        dx = dx + residual.double()
        bx = bx + U * (dx.abs() + residual.double().abs())
    depth = T / 100 + 100
    dw, db = (dy * h).sum(0), dy.sum(0)
    return (dx, bx), (dw, (depth + 4) * U * (dy * h).abs().sum(0)), (db, depth * U * dy.abs().sum(0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_forward(rows, cols, pad, offset, dtype):
    _, ld, x, w, b = _inputs(rows, cols, pad, offset, dtype, 1)
    y, buf = lu.empty_matrix(rows, cols, dtype, ld, offset)
    mean, rstd = torch.full((rows + 8,), float("nan"), device="cuda"), torch.full((rows + 8,), float("nan"), device="cuda")
    fs.fsdp_layernorm_forward(x, y, w, b, mean[:rows], rstd[:rows], EPS)
    fs.fsdp_check_status()
    (wy, by), (wm, bm), (wr, br) = forward64(x, w, b)
    lu.check(y, wy, by, "y")
    lu.check(mean[:rows], wm, bm, "mean")
    lu.check(rstd[:rows], wr, br, "rstd")
    assert lu.untouched(y, buf) and mean[rows:].isnan().all() and rstd[rows:].isnan().all()
    # without the parts that may be left out, and in place
    fs.fsdp_layernorm_forward(x, y, eps=EPS)
    (wy, by), _, _ = forward64(x, None, None)
    lu.check(y, wy, by, "y without weight and bias")
    fs.fsdp_layernorm_forward(x, x, eps=EPS)
    assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_of_rows_far_from_zero(dtype):
    """A row's own offset, 4096 times its spread, costs no digits of what is left."""
    g = lu.gen(3)
    for cols in (200, 2048, 9000):
        x = (torch.randint(-128, 129, (33, cols), generator=g, device="cuda").float() / 128 + 4096.0).to(F32)
        x = x.to(dtype)
        y, mean, rstd = torch.empty_like(x), torch.empty(33, device="cuda"), torch.empty(33, device="cuda")
        fs.fsdp_layernorm_forward(x, y, mean=mean, rstd=rstd, eps=EPS)
        (wy, by), (wm, bm), (wr, br) = forward64(x, None, None)
        lu.check(y, wy, by, "y")
        lu.check(rstd, wr, br, "rstd")
        assert (mean.double() - wm).abs().max() <= U * 4097 + bm.max()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [24, 200, 1001, 2048, 9000])
def test_forward_of_rows_that_begin_elsewhere(cols, dtype):
    """The first columns of some rows say nothing about the rest."""
    g, _, x, w, b = _inputs(50, cols, 0, 0, dtype, 12)
    x[::3, :8] = 100.0
    x[1::3, 0] = -3000.0
    x[5] = 7.25
    y, mean, rstd = torch.empty_like(x), torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    fs.fsdp_layernorm_forward(x, y, w, b, mean, rstd, EPS)
    (wy, by), (wm, bm), (wr, br) = forward64(x, w, b)
    lu.check(y, wy, by, "y")
    lu.check(mean, wm, bm, "mean")
    lu.check(rstd, wr, br, "rstd")
    assert mean[5] == 7.25


@pytest.mark.parametrize("dtype,grad_dtype,accumulate", [(BF16, BF16, False), (BF16, F32, True), (F32, F32, False), (F32, F32, True),
                                                         (F32, BF16, False), (BF16, BF16, True)])
@pytest.mark.parametrize("rows,cols,pad,offset", SHAPES)
def test_backward(rows, cols, pad, offset, dtype, grad_dtype, accumulate):
    g, ld, x, w, _ = _inputs(rows, cols, pad, offset, dtype, 2)
    dy = lu.matrix(rows, cols, dtype, 1e-3, g, ld, offset)
    residual = lu.matrix(rows, cols, dtype, 1e-3, g, ld, offset)
    mean, rstd = x.double().mean(1).float(), ((x.double().var(1, unbiased=False) + EPS) ** -0.5).float()
    dx, buf = lu.empty_matrix(rows, cols, dtype, ld, offset)
    dwb, wbuf = lu.empty_matrix(2, cols, grad_dtype, cols + 5, offset)
    dw, db = dwb[0], dwb[1]
    old = torch.randn(2, cols, generator=g, device="cuda").to(grad_dtype) * 1e-2
    if accumulate:
        dwb.copy_(old)
    n = fs.fsdp_layernorm_workspace_bytes(rows, cols)
    ws = torch.full((n // 4 + 8,), float("nan"), device="cuda")      # no initial contents needed, nothing behind it written
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, dx, w, dw, db, residual, accumulate, ws[:n // 4])
    fs.fsdp_check_status()
    (wx, bx), (ww, bw), (wb, bb) = backward64(dy, x, mean, rstd, w, residual)
    lu.check(dx, wx, bx, "dx")
    if accumulate:
        ww, wb = ww + old[0].double(), wb + old[1].double()
        bw, bb = bw + U * ww.abs(), bb + U * wb.abs()
    lu.check(dw, ww, bw, "dw")
    lu.check(db, wb, bb, "db")
    assert lu.untouched(dx, buf) and lu.untouched(dwb, wbuf) and ws[n // 4:].isnan().all()
    # dx into the residual's own buffer, and, without weight or residual, into dy's and x's own
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, residual, w, residual=residual)
    assert torch.equal(residual, dx)
    plain, _ = lu.empty_matrix(rows, cols, dtype, ld, offset)
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, plain)
    (wx, bx), _, _ = backward64(dy, x, mean, rstd, None, None)
    lu.check(plain, wx, bx, "dx alone")
    keep = dy.clone()
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, dy)
    assert torch.equal(plain, dy)
    dy.copy_(keep)
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, x)
    assert torch.equal(plain, x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(500, 64), (700, 333), (333, 1001), (129, 4096), (40, 9000)])
def test_matrices_out_of_step(rows, cols, dtype):
    """Matrices whose rows start at different addresses modulo 16."""
    g = lu.gen(21)
    places = [(cols, 0), (cols + 1, 0), (cols, 3), (cols + 5, 1)]
    x0 = (torch.randn(rows, cols, generator=g, device="cuda") + 0.5).to(dtype)
    dy0, r0 = ((torch.randn(rows, cols, generator=g, device="cuda") * 1e-3).to(dtype) for _ in range(2))
    w, b = (torch.randn(cols, generator=g, device="cuda").to(dtype) for _ in range(2))

    def put(v, k):
        m, buf = lu.empty_matrix(rows, cols, dtype, *places[k % 4])
        m.copy_(v)
        return m, buf

    def bounds(y, mean, rstd, dx, dw, db):
        (wy, by), (wm, bm), (wr, br) = forward64(x0, w, b)
        lu.check(y, wy, by, "y")
        (wx, bx), (ww, bw), (wb, bb) = backward64(dy0, x0, mean, rstd, w, r0)
        lu.check(dx, wx, bx, "dx")
        lu.check(dw, ww, bw, "dw")
        lu.check(db, wb, bb, "db")

    ws = torch.empty(fs.fsdp_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    for turn in range(4):
        x, _ = put(x0, turn)
        y, ybuf = put(torch.full_like(x0, float("nan")), turn + 1)
        mean, rstd, sums = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(2, cols, device="cuda")
        fs.fsdp_layernorm_forward(x, y, w, b, mean, rstd, EPS)
        dx, xbuf = put(torch.full_like(x0, float("nan")), turn + 2)
        fs.fsdp_layernorm_backward(put(dy0, turn + 3)[0], x, mean, rstd, dx, w, sums[0], sums[1], put(r0, turn + 1)[0], workspace=ws)
        bounds(y, mean, rstd, dx, sums[0], sums[1])
        assert lu.untouched(y, ybuf) and lu.untouched(dx, xbuf)
    fs.fsdp_check_status()


@pytest.mark.parametrize("which", ["dw", "db"])
def test_one_sum_alone(which):
    g, _, x, w, _ = _inputs(100, 96, 0, 0, BF16, 5)
    dy = lu.matrix(100, 96, BF16, 1e-3, g)
    mean, rstd = x.double().mean(1).float(), ((x.double().var(1, unbiased=False) + EPS) ** -0.5).float()
    ws = torch.empty(fs.fsdp_layernorm_workspace_bytes(100, 96), dtype=torch.uint8, device="cuda")
    both = torch.empty(2, 96, device="cuda")
    dx, one = torch.empty_like(x), torch.empty(96, device="cuda")
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, dx, w, both[0], both[1], workspace=ws)
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, dx, w, workspace=ws, **{which: one})
    assert torch.equal(one, both[0] if which == "dw" else both[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [40, 200, 768, 1001, 2048, 11008, 12000, 20480])
def test_bad_rows_stay_alone(cols, dtype):
    """Infinities and NaNs make their own row NaN, in y and in dx, and no other."""
    g, _, x, w, b = _inputs(9, cols, 0, 0, dtype, 6)
    dy = lu.matrix(9, cols, dtype, 1e-3, g)
    y0, dx0, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    fs.fsdp_layernorm_forward(x, y0, w, b, mean, rstd, EPS)
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, dx0, w)
    x[2, cols // 2], x[5, 0], x[7, cols - 1] = float("inf"), float("nan"), -float("inf")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    m, r = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    fs.fsdp_layernorm_forward(x, y, w, b, m, r, EPS)
    fs.fsdp_layernorm_backward(dy, x, m, r, dx, w)
    good = [0, 1, 3, 4, 6, 8]
    assert torch.equal(y[good], y0[good]) and torch.equal(dx[good], dx0[good])
    assert y[[2, 5, 7]].isnan().all() and dx[[2, 5, 7]].isnan().all() and r[[2, 5, 7]].isnan().all()


def test_constant_rows():
    """No spread: y is the bias, and rstd that of eps alone."""
    x = torch.full((4, 300), 1e4, device="cuda")
    b = torch.randn(300, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    fs.fsdp_layernorm_forward(x, y, None, b, mean, rstd, EPS)
    assert torch.equal(y, b.expand(4, -1)) and (mean == 1e4).all()
    assert ((rstd.double() - EPS ** -0.5).abs() <= 4 * U * EPS ** -0.5 + 2.0 ** -20).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=BF16)
    s = torch.empty(0, device="cuda")
    fs.fsdp_layernorm_forward(x, x, mean=s, rstd=s)
    dw, db = torch.full((64,), float("nan"), device="cuda"), torch.full((64,), float("nan"), device="cuda")
    fs.fsdp_layernorm_backward(x, x, s, s, x, dw=dw, db=db)
    assert not dw.any() and not db.any()
    dw.fill_(3.0)
    fs.fsdp_layernorm_backward(x, x, s, s, x, dw=dw, accumulate=True)
    assert (dw == 3.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_against_differences(dtype):
    """Directional derivatives of sum(y v) in x, weight and bias: the kernel's gradients against
    central differences of the definition in 64 bits."""
    g, _, x, w, b = _inputs(13, 130, 0, 0, dtype, 8)
    v = lu.matrix(13, 130, dtype, 1.0, g)
    y, mean, rstd = torch.empty_like(x), torch.empty(13, device="cuda"), torch.empty(13, device="cuda")
    fs.fsdp_layernorm_forward(x, y, w, b, mean, rstd, EPS)
    dx, dw, db = torch.empty_like(x), torch.empty(130, device="cuda"), torch.empty(130, device="cuda")
    ws = torch.empty(fs.fsdp_layernorm_workspace_bytes(13, 130), dtype=torch.uint8, device="cuda")
    fs.fsdp_layernorm_backward(v, x, mean, rstd, dx, w, dw, db, workspace=ws)

    def value(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return ((d * (d.square().mean(1, keepdim=True) + EPS) ** -0.5 * w + b) * v.double()).sum()

    a = [x.double(), w.double(), b.double()]
    for k, got in ((0, dx), (1, dw), (2, db)):
        t = torch.randn(a[k].shape, generator=g, device="cuda").double()
        e = 1e-5
        up, down = list(a), list(a)
        up[k], down[k] = a[k] + e * t, a[k] - e * t
        want = float((value(*up) - value(*down)) / (2 * e))
        size = float((got.double() * t).square().sum().sqrt())
        # the gradient's elements carry independent roundings of its type, the differences 1e-9
        tol = 6 * lu.OUT_ULP[got.dtype] * size + 200 * U * size * 13 ** 0.5 + 1e-6 * size + 1e-9
        assert abs(float((got.double() * t).sum()) - want) <= tol


def test_rows_past_32_bits():
    """Rows whose offsets pass 2^32 elements."""
    ld, cols = (1 << 31) - 2048, 4096
    buf = torch.empty(2 * ld + cols, dtype=BF16, device="cuda")
    x = buf.as_strided((3, cols), (ld, 1))
    small = torch.randn(3, cols, generator=lu.gen(9), device="cuda").to(BF16)
    x.copy_(small)
    want, dy, dx = torch.empty_like(small), torch.randn(3, cols, generator=lu.gen(10), device="cuda").to(BF16), torch.empty_like(small)
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    fs.fsdp_layernorm_forward(small, want, mean=mean, rstd=rstd)
    fs.fsdp_layernorm_backward(dy, small, mean, rstd, dx)
    far = torch.empty_like(small)
    fs.fsdp_layernorm_backward(dy, x, mean, rstd, far)
    assert torch.equal(far, dx)
    fs.fsdp_layernorm_forward(x, x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("rows,cols", [(3000, 1024), (5000, 200), (700, 12000), (250, 20480)])
def test_same_bits_on_two_streams_and_in_a_graph(rows, cols):
    """Two calls at once with workspaces of their own, and a captured pair replayed on new inputs."""
    g, _, x, w, b = _inputs(rows, cols, 0, 0, BF16, 11)
    dy = lu.matrix(rows, cols, BF16, 1e-3, g)
    n = fs.fsdp_layernorm_workspace_bytes(rows, cols)

    def call(out):
        fs.fsdp_layernorm_forward(x, out["y"], w, b, out["mean"], out["rstd"], EPS)
        fs.fsdp_layernorm_backward(dy, x, out["mean"], out["rstd"], out["dx"], w, out["dw"], out["db"], workspace=out["ws"])

    def buffers():
        return dict(y=torch.empty_like(x), mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"),
                    dx=torch.empty_like(x), dw=torch.empty(cols, device="cuda"), db=torch.empty(cols, device="cuda"),
                    ws=torch.empty(n, dtype=torch.uint8, device="cuda"))

    def same(p, q):
        return all(torch.equal(p[k], q[k]) for k in p if k != "ws")

    want, outs = buffers(), [buffers(), buffers()]
    call(want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, out in zip(streams, outs):
            with torch.cuda.stream(st):
                call(out)
    torch.cuda.synchronize()
    assert same(want, outs[0]) and same(want, outs[1])
    graph, out = torch.cuda.CUDAGraph(), buffers()
    with torch.cuda.graph(graph):
        call(out)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda").to(BF16))
    graph.replay()
    call(want)
    torch.cuda.synchronize()
    assert same(want, out)
