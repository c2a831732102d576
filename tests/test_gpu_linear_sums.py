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


def product(mode, R, C, grad_dtype=None):
    """out[r][c] = sum over k of R[r][k] C[c][k] by one of the three calls, and the same in 64 bits."""
    K, dtype = R.shape[1], R.dtype
    out, buf = lu.empty_matrix(R.shape[0], C.shape[0], grad_dtype or dtype)
    if mode == "forward":
        fs.fsdp_linear_forward(R, C, out, workspace=lu.workspace(R.shape[0], K, C.shape[0], dtype))
    elif mode == "dgrad":
        fs.fsdp_linear_dgrad(R, C.t().contiguous(), out, workspace=lu.workspace(R.shape[0], C.shape[0], K, dtype))
    else:
        fs.fsdp_linear_wgrad(R.t().contiguous(), C.t().contiguous(), out, workspace=lu.workspace(K, C.shape[0], R.shape[0], dtype))
    fs.fsdp_check_status()
    assert lu.untouched(out, buf)
    return out, R.double() @ C.double().t()


# mode, rows and columns of the result, K: CTA pairs with whole tiles of 256 columns, with halved
# ones in the last wave, and of 128 columns; split tiles; slabs of rows; the FMA units
SIZES = [("forward", 2432, 1792, 2048), ("forward", 2600, 2500, 2048), ("forward", 1000, 2048, 2048), ("forward", 300, 1000, 2048),
         ("forward", 600, 700, 16384), ("forward", 64, 4096, 512), ("dgrad", 2300, 2048, 2304), ("dgrad", 2600, 2500, 2048),
         ("dgrad", 1000, 2048, 2048), ("dgrad", 300, 2048, 1000), ("dgrad", 600, 700, 16384), ("dgrad", 100, 700, 1500),
         ("wgrad", 2048, 2048, 2048), ("wgrad", 2500, 2600, 2048), ("wgrad", 1000, 2048, 300), ("wgrad", 500, 600, 16384),
         ("wgrad", 2600, 1300, 16384), ("wgrad", 128, 128, 16384)]
ON_FMA = [("forward", 300, 200, 256), ("forward", 3, 2048, 2048), ("dgrad", 300, 200, 256), ("dgrad", 3, 2048, 2048),
          ("wgrad", 32, 64, 16384), ("wgrad", 300, 200, 256)]


@pytest.mark.parametrize("mode,rows,cols,K,dtype", [(*s, F32) for s in SIZES + ON_FMA] + [(*s, BF16) for s in SIZES if s[0] == "wgrad"])
def test_relative_error_of_fp32_results(mode, rows, cols, K, dtype):
    """In norm, 2e-6: the accumulators are added to fp32 registers after 8 steps of 16 products at
    full magnitude (fp32 operands; the other term products are smaller by 2^-8) or 32 (bf16), of
    which each rounds the growing sum towards zero by at most 2^-23, on average half of it, and the
    parts' errors have the signs of the parts: 32 * 2^-24 * 2 / 3 = 1.3e-6; dropped term products below
    2^-24 of each product, 3 of them, and sums of up to 128 parts, sqrt(128) * 2^-24, in all 2e-6.
    Without the three smallest of the products that are kept, (0,2), (2,0) and (1,1), 3e-6."""
    g = lu.gen(81)
    out, want = product(mode, lu.matrix(rows, K, dtype, 1.0, g), lu.matrix(cols, K, dtype, 1.0, g), F32)
    assert (out.double() - want).norm() <= 2e-6 * want.norm()


def carried_by(plane, rows, K, other, g):
    """fp32 rows of K = 4 j elements a + m + l, hi + mid + lo terms of known magnitudes, that cancel
    along k against those of carried_by(.., other=True) but for what one pair of planes carries:
      lo   x = a + m + s l, -(a + m), ..      other = b, b, ..
      mid  x = a + s m, -a, -(a + s m), a     other = b + t n, b + t n, b, b
    with a sign s (t) to each row and each 64 elements."""
    def pick(shape, values):
        return torch.tensor(values, device="cuda", dtype=F32)[torch.randint(len(values), shape, generator=g, device="cuda")]

    sign = pick((rows, K // 64), [-1.0, 1.0]).repeat_interleave(16, 1)
    a = pick((rows, K // 4), [1.25, 1.375])
    m = pick((rows, K // 4), [1.0, 1.25, 1.5, 1.75]) * 2.0 ** -9
    low = pick((rows, K // 4), [1.0, 1.25, 1.5, 1.75]) * 2.0 ** -18
    if plane == "lo":
        four = [a] * 4 if other else [a + m + sign * low, -(a + m)] * 2
    else:
        four = [a + sign * m] * 2 + [a] * 2 if other else [a + sign * m, -a, -(a + sign * m), a]
    return torch.stack(four, -1).reshape(rows, K).contiguous()


@pytest.mark.parametrize("mode,rows,cols,K", SIZES)
@pytest.mark.parametrize("planes", ["lo x hi", "hi x lo", "mid x mid"])
def test_low_planes_carry_the_result(mode, rows, cols, K, planes):
    """Each of the three smallest products kept, (2,0), (0,2) and (1,1), by itself the result.
    The terms' products below 2 cancel inside a step of 16, each such step shifts the sum by at
    most two units of 2^-23 (of linear_util's bound): 2^-26 K.  A stage of 64 elements is worth
    32 * 1.25 * 2^-18 (lo) or 16 * 2^-18 (mid) at least, with a sign of its own: at K = 2048 twice
    that, what a stage with the planes of another would be off by, is above the bound."""
    K -= K % 64
    g = lu.gen(82)
    plane = "mid" if planes == "mid x mid" else "lo"
    x, y = carried_by(plane, rows, K, False, g), carried_by(plane, cols, K, True, g)
    if planes == "hi x lo":
        x, y = carried_by(plane, rows, K, True, g), carried_by(plane, cols, K, False, g)
    out, want = product(mode, x, y)
    err = (out.double() - want).abs().max().item()
    assert err <= K * 2.0 ** -26, f"{err / (K * 2.0 ** -26):.3g} of the bound"
    assert want.abs().max() > 4 * K * 2.0 ** -26


@pytest.mark.parametrize("rows,cin,cout", [(1000, 2048, 2048), (70, 500, 900), (64, 96, 80), (3, 700, 300)])
def test_infinities_of_fp32_operands(rows, cin, cout):
    """CTA pairs, split tiles, small products and few rows: what depends on an infinity is not
    finite (it may be a NaN), the rest is as without it, and a dropped element is 0."""
    g = lu.gen(83)
    x, w, dz = (lu.matrix(r, c, F32, 1.0, g) for r, c in ((rows, cin), (cout, cin), (rows, cout)))
    spec = fs.DropoutSpec(0.3, 8)
    ws = lu.workspace(rows, cin, cout, F32)

    def run(x, dz):
        y, dx, dw, db = (torch.empty(s, device="cuda") for s in ((rows, cout), (rows, cin), (cout, cin), (cout,)))
        fs.fsdp_linear_forward(x, w, y, dropout=spec, workspace=ws)
        fs.fsdp_linear_dgrad(dz, w, dx, workspace=ws)
        fs.fsdp_linear_wgrad(dz, x, dw, db, workspace=ws)
        fs.fsdp_check_status()
        return y, dx, dw, db

    clean = run(x, dz)
    xi, zi = x.clone(), dz.clone()
    xi[2, 7], zi[1, 5] = float("inf"), float("-inf")
    y, dx, dw, db = run(xi, zi)
    keep = lu.keep_mask(rows, cout, spec)
    assert not y[2][keep[2]].isfinite().any() and (y[2][~keep[2]] == 0).all()
    assert not dx[1].isfinite().any() and not dw[5].isfinite().any() and not dw[:, 7].isfinite().any()
    assert not db[5].isfinite()
    for got, want, without in ((y, clean[0], (2, None)), (dx, clean[1], (1, None)), (dw, clean[2], (5, 7))):
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[without[0]] = False
        if without[1] is not None:
            rest[:, without[1]] = False
        assert torch.equal(got[rest], want[rest])
    assert torch.equal(db[torch.arange(cout) != 5], clean[3][torch.arange(cout) != 5])
