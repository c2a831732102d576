"""Newton-Schulz orthogonalisation against its definition in 64 bits (bounds: ns_util)."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu
import ns_util as nu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# vectors, tiles and their edges in both orientations, sides of no 16-byte multiple, a long thin
# matrix (K split over clusters), several tiles of each configuration
SHAPES = [(1, 1), (1, 7), (5, 3), (64, 32), (33, 65), (64, 64), (65, 64), (128, 128), (127, 129), (200, 1000), (256, 256), (257, 130),
          (384, 640), (16, 16384), (9000, 24), (512, 2048), (1001, 777), (1024, 1024), (1300, 2600), (3000, 1100),
          (700, 6000), (64, 60000), (3, 1200), (30, 500), (31, 29), (64, 110), (64, 120), (8, 2000), (61, 63), (2, 2), (64, 256), (128, 96), (100, 120), (90, 97)]


def workspace(count, rows, cols, extra=64):
    """Scratch with NaN in it, and behind it a stretch that nothing may write."""
    n = fs.fsdp_newton_schulz_workspace_bytes(count, rows, cols)
    buf = torch.full((n // 4 + extra,), float("nan"), device="cuda")
    return buf[:n // 4], buf[n // 4:]


@pytest.mark.parametrize("src_dtype,dst_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_matrix(rows, cols, src_dtype, dst_dtype):
    g = lu.gen(rows * 31 + cols)
    x = nu.gradient(rows, cols, g, dtype=src_dtype)
    y, buf = lu.empty_matrix(rows, cols, dst_dtype)
    ws, behind = workspace(1, rows, cols)
    fs.fsdp_newton_schulz(x, y, workspace=ws)
    fs.fsdp_check_status()
    nu.check(y, x)
    assert lu.untouched(y, buf) and behind.isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,pad,offset", [(40, 72, 8, 0), (72, 40, 3, 1), (130, 257, 1, 3), (300, 140, 0, 5)])
def test_strides_and_offsets_and_in_place(rows, cols, pad, offset, dtype):
    g = lu.gen(7)
    x = lu.matrix(rows, cols, dtype, 1e-3, g, cols + pad, offset)
    y, buf = lu.empty_matrix(rows, cols, dtype, cols + pad + 2, offset)
    ws, _ = workspace(1, rows, cols)
    fs.fsdp_newton_schulz(x, y, workspace=ws)
    nu.check(y, x)
    assert lu.untouched(y, buf)
    whole = torch.as_strided(x, (x.untyped_storage().nbytes() // x.element_size(),), (1,), 0)
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask.as_strided(x.shape, x.stride(), x.storage_offset()).fill_(False)
    fs.fsdp_newton_schulz(x, x, workspace=ws)
    assert torch.equal(x, y) and whole[mask].isnan().all()


@pytest.mark.parametrize("count,rows,cols", [(2, 64, 32), (5, 100, 300), (70, 48, 64), (12, 300, 300), (3, 1024, 600)])
def test_batches(count, rows, cols):
    """Batches of matrices of all magnitudes; more than 64, or more than the workspace takes at once,
    pass in parts; the same bits again."""
    g = lu.gen(count)
    xs = [nu.gradient(rows, cols, g) * 10.0 ** (i % 7 - 3) for i in range(count)]
    ys = [torch.empty_like(x) for x in xs]
    ws, behind = workspace(count, rows, cols)
    fs.fsdp_newton_schulz(xs, ys, workspace=ws)
    fs.fsdp_check_status()
    for i in (0, 1, count // 2, count - 1):
        nu.check(ys[i], xs[i], f"matrix {i}")
    assert behind.isnan().all()
    again = [torch.empty_like(x) for x in xs]
    fs.fsdp_newton_schulz(xs, again, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(ys, again))


@pytest.mark.parametrize("coeffs", [[(1.5, -0.5, 0.0)] * 12, [(15 / 8, -10 / 8, 3 / 8)] * 9, [(3.4445, -4.7750, 2.0315)],
                                    [(8.28721201814563, -23.595886519098837, 17.300387312530933),
                                     (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
                                     (3.9486908534822946, -2.908902115962949, 0.5518191394370137)], [(0.0, 0.0, 0.0)] * 2])
def test_schedules(coeffs):
    g = lu.gen(5)
    x = nu.gradient(150, 220, g, rank=8)
    y = torch.empty_like(x)
    ws, _ = workspace(1, 150, 220)
    fs.fsdp_newton_schulz(x, y, steps=len(coeffs), coeffs=coeffs, workspace=ws)
    nu.check(y, x, steps=len(coeffs), coeffs=coeffs)


def test_singular_values():
    """From orthogonal factors: every singular value of |G| / 100 and more comes out in [0.68, 1.21],
    and the singular vectors stay."""
    g = lu.gen(6)
    u, _ = torch.linalg.qr(torch.randn(200, 160, generator=g, device="cuda").double())
    v, _ = torch.linalg.qr(torch.randn(300, 160, generator=g, device="cuda").double())
    s = torch.logspace(0, -1.2, 160, device="cuda").double()
    s = s / s.norm()
    assert float(s.min()) >= 0.01
    x = ((u * s) @ v.t()).float()
    y = torch.empty_like(x)
    ws, _ = workspace(1, 200, 300)
    fs.fsdp_newton_schulz(x, y, workspace=ws)
    core = u.t() @ y.double() @ v
    d = torch.diagonal(core)
    assert 0.68 <= float(d.min()) and float(d.max()) <= 1.21
    assert float((core - torch.diag(d)).norm()) <= 1e-4 * float(d.norm())


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e12])
def test_small_and_large_norms(scale):
    """The norm divides out; below eps the matrix is divided by eps."""
    g = lu.gen(8)
    x = nu.gradient(96, 80, g) * scale
    y = torch.empty_like(x)
    ws, _ = workspace(1, 96, 80)
    fs.fsdp_newton_schulz(x, y, workspace=ws)
    nu.check(y, x.double(), eps=1e-7)


@pytest.mark.parametrize("rows,cols", [(32, 48), (300, 520)])
def test_bad_matrices_stay_alone(rows, cols):
    g = lu.gen(9)
    xs = [nu.gradient(rows, cols, g) for _ in range(5)]
    ws, _ = workspace(5, rows, cols)
    want = [torch.empty_like(x) for x in xs]
    fs.fsdp_newton_schulz(xs, want, workspace=ws)
    xs[1].zero_()
    xs[2][rows // 2, 3], xs[3][0, cols - 1] = float("nan"), float("inf")
    ys = [torch.empty_like(x) for x in xs]
    fs.fsdp_newton_schulz(xs, ys, workspace=ws)
    fs.fsdp_check_status()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[4], want[4])
    assert not ys[1].any() and ys[2].isnan().all()
    assert (ys[3].isnan() | (ys[3] == 0)).all() and ys[3].isnan().any()


def test_rows_past_32_bits():
    """A source and a destination whose row offsets pass 2^32 elements."""
    ld, cols = (1 << 31) - 2048, 300
    buf = torch.empty(2 * ld + cols, dtype=BF16, device="cuda")
    x = buf.as_strided((3, cols), (ld, 1))
    small = nu.gradient(3, cols, lu.gen(10), dtype=BF16)
    x.copy_(small)
    y, z = torch.empty_like(small), torch.empty_like(small)
    ws, _ = workspace(1, 3, cols)
    fs.fsdp_newton_schulz(small, y, workspace=ws)
    fs.fsdp_newton_schulz(x, z, workspace=ws)
    assert torch.equal(y, z)
    fs.fsdp_newton_schulz(x, x, workspace=ws)
    assert torch.equal(x, y)


def test_two_streams_and_a_graph():
    """Two calls at once with workspaces of their own; a captured call replayed on new inputs; two
    captured calls that share a workspace, one after the other."""
    g = lu.gen(11)
    xs = [nu.gradient(500, 700, g) for _ in range(3)]
    want = [torch.empty_like(x) for x in xs]
    spaces = [workspace(1, 500, 700)[0] for _ in range(3)]
    for x, y in zip(xs, want):
        fs.fsdp_newton_schulz(x, y, workspace=spaces[0])
    ys = [torch.empty_like(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                fs.fsdp_newton_schulz(xs[i], ys[i], workspace=spaces[i])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
    a, b = xs[0].clone(), xs[1].clone()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for graph, x, y in zip(graphs, (a, b), ys):
        with torch.cuda.graph(graph):
            fs.fsdp_newton_schulz(x, y, workspace=spaces[2])
    for graph in graphs:
        graph.replay()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
    a.copy_(xs[2])
    graphs[0].replay()
    assert torch.equal(ys[0], want[2])
    fs.fsdp_check_status()


# Every product's operands are held to 2^-22 of themselves.  What a step makes of an error e of X X^T in the directions
# at the top is the polynomial's terms over its sum, (3.44 + 4.78 t + 2.03 t^2) / p(s) s, at most 12 / 0.7 e; the last
# step adds its own, the one before it as much again, and those before are pulled together: 2 x 17 x 2^-22.
IN_NORM = 2 * 12 / 0.7 * 2.0 ** -22


@pytest.mark.parametrize("count,rows,cols", [(1, 173, 6644), (1, 8000, 128), (12, 320, 1280), (8, 384, 2176), (1, 3456, 32), (2, 640, 2000),
                                             (1, 800, 2400)])
def test_error_in_norm_of_long_matrices(count, rows, cols):
    """Where steps share a pass over X, what A loses by it must not show."""
    g = lu.gen(rows + cols)
    xs = [nu.gradient(rows, cols, g) for _ in range(count)]
    ys = [torch.empty_like(x) for x in xs]
    fs.fsdp_newton_schulz(xs, ys, workspace=workspace(count, rows, cols)[0])
    for x, y in zip(xs, ys):
        want = nu.steps_in(x, torch.float64)
        assert float((y.double() - want).norm()) <= IN_NORM * float(want.norm())
