"""Layer norm of rows far from zero in which few elements deviate: the others' results are small
beside the spread, and the mean's rounding to fp32 must not show in them.  Bounds: those of
test_gpu_layernorm."""
import pytest
import torch

import fsdp_sharded_state_gb300 as fs

import linear_util as lu
from test_gpu_layernorm import BF16, EPS, F32, forward64

pytestmark = pytest.mark.gpu

# every way a row is spread over threads, whole chunks and single columns
COLS = [24, 61, 120, 200, 255, 512, 1001, 2048, 4096, 4097, 6144, 8192, 11008, 16384, 16385, 20480, 65536]


def check(x, w=None, b=None):
    rows = x.shape[0]
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    fs.fsdp_layernorm_forward(x, y, w, b, mean, rstd, EPS)
    fs.fsdp_check_status()
    (wy, by), (wm, bm), (wr, br) = forward64(x, w, b)
    lu.check(y, wy, by, "y")
    lu.check(mean, wm, bm, "mean")
    lu.check(rstd, wr, br, "rstd")
    return y, mean, rstd


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_few_elements_deviate(cols, dtype):
    """Offsets of several sizes, one to five elements one or three bf16 steps or a half of it away."""
    g = lu.gen(31)
    x = torch.empty(60, cols, device="cuda")
    for r in range(60):
        c = (4992.0, -4992.0, 1.0078125, 7e4, -0.0123291015625, 250.0)[r % 6]
        x[r] = c
        at = torch.randperm(cols, generator=g, device="cuda")[:1 + r % 5]
        x[r, at] = c * (1 + (2.0 ** -7, 3 * 2.0 ** -7, -0.5)[r // 6 % 3])
    x = x.to(dtype)
    assert (x.amax(1) > x.amin(1)).all()          # the deviations survive the rounding to the type
    check(x)


@pytest.mark.parametrize("cols", COLS)
def test_means_of_all_sizes(cols):
    """Means from none to a hundred times the spread, in neighbouring rows: those that are corrected
    beside those that need not be."""
    g = lu.gen(32)
    factor = torch.tensor([0.0, 0.5, 1.0, 2.0, 3.5, 3.9, 4.1, 5.0, 8.0, 30.0, 100.0], device="cuda").repeat(6)[:, None]
    x = (torch.randn(66, cols, generator=g, device="cuda") + factor).to(BF16)
    w, b = torch.randn(cols, generator=g, device="cuda").to(BF16), torch.randn(cols, generator=g, device="cuda").to(BF16)
    y, mean, rstd = check(x, w, b)
    # a row's bits do not depend on the rows around it
    order = torch.randperm(66, generator=g, device="cuda")
    y2, mean2, rstd2 = check(x[order].contiguous(), w, b)
    assert torch.equal(y2, y[order]) and torch.equal(mean2, mean[order]) and torch.equal(rstd2, rstd[order])


@pytest.mark.parametrize("cols", [40, 1001, 4096, 20480])
def test_bad_rows_beside_far_ones(cols):
    """Infinities, NaNs, constant rows and rows of zeros in every second row, in place."""
    g = lu.gen(33)
    x = torch.full((24, cols), 4992.0, device="cuda")
    x[:, cols // 3] = 5024.0
    want = torch.empty(24, cols, dtype=BF16, device="cuda")
    fs.fsdp_layernorm_forward(x.to(BF16), want, eps=EPS)
    x[1], x[3], x[5, cols - 1], x[7, 0], x[9] = 0.0, 4992.0, float("inf"), float("nan"), torch.randn(cols, generator=g, device="cuda")
    y = x.to(BF16)
    fs.fsdp_layernorm_forward(y, y, eps=EPS)
    fs.fsdp_check_status()
    rest = [r for r in range(24) if r not in (1, 3, 5, 7, 9)]
    assert torch.equal(y[rest], want[rest]) and y[[5, 7]].isnan().all() and not y[[1, 3]].any() and y[9].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [40, 1001, 4096, 20480])
def test_finite_rows_beyond_the_range(cols, dtype):
    """A sum beyond fp32's range makes its row NaN; differences whose squares are beyond it make rstd 0 and y the
    bias; a constant row of large values is exact.  The rows between them are as they are alone."""
    g = lu.gen(34)
    x = torch.randn(9, cols, generator=g, device="cuda").to(dtype)
    b = torch.randn(cols, generator=g, device="cuda").to(dtype)
    want, y = torch.empty_like(x), torch.empty_like(x)
    fs.fsdp_layernorm_forward(x, want, None, b, eps=EPS)
    sign = torch.where(torch.arange(cols, device="cuda") % 2 == 0, 1.0, -1.0)
    x[1], x[3], x[5] = 3e38, (1e20 * sign).to(dtype), 2.0 ** 60
    x[7] = (1e30 * (1 + 0.25 * sign)).to(dtype)
    mean, rstd = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    fs.fsdp_layernorm_forward(x, y, None, b, mean, rstd, EPS)
    fs.fsdp_check_status()
    assert y[1].isnan().all() and torch.equal(y[[3, 5, 7]], b.expand(3, -1))
    assert (rstd[[3, 7]] == 0).all() and mean[5] == 2.0 ** 60
    assert torch.equal(y[::2], want[::2])
