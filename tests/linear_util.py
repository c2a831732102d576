"""Definitions of the layer operators in 64 bits, and the error bounds of their tests.

The bounds follow from how a result is formed.  With M = sum over k of |a_k b_k|:
  - one product step of the tensor cores adds a group of 16 products to an fp32
    accumulator; aligning the group and rounding the sum lose at most two units in the last
    place of a magnitude below M, 2 * 2^-23 M.  K products take K / 16 steps (a few more
    where ragged K is padded): bf16 operands, (K / 16 + 8) * 2^-22 M;
  - fp32 operands as three bf16 terms: the dropped term products are below 2^-22 of each
    product; the accumulators hold at most 256 products per plane pair, six pairs, before they
    are added in fp32: (6 * 16 + 8 + K / 256) * 2^-22 M;
  - the epilogue is fp32: a few roundings of 2^-24 and CUDA's erff and expf (2 ulp), together
    below 2^-20 of the largest intermediate magnitude;
  - one rounding to the output type: the unit roundoff 2^-8 (bf16, 8 significant bits) or 2^-24 (fp32) of the result.
"""
import numpy as np
import torch

import fsdp_sharded_state_gb300 as fs

OUT_ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def product_bound(K, M, dtype):
    n = K / 16 + 8 if dtype == torch.bfloat16 else 6 * 16 + 8 + K / 256
    return n * 2.0 ** -22 * M


def philox_words(rows, cols, seed, layer, row0=0):
    """uint64 array [rows][cols] of the generator's words, from the published round function."""
    nq = (cols + 3) // 4
    r = np.repeat(np.arange(row0, row0 + rows, dtype=np.uint64), nq)
    c = [np.tile(np.arange(nq, dtype=np.uint64), rows), r & np.uint64(0xFFFFFFFF), r >> np.uint64(32),
         np.full(rows * nq, layer, np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    lo, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> sh) ^ c[1] ^ np.uint64(k0), q & lo, (p >> sh) ^ c[3] ^ np.uint64(k1), p & lo]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1).reshape(rows, 4 * nq)[:, :cols]


def keep_mask(rows, cols, spec, device="cuda"):
    w = philox_words(rows, cols, spec.seed, spec.layer, spec.row0)
    return torch.from_numpy(w >= np.uint64(int(spec.p * 2.0 ** 32))).to(device)


def drop64(v, spec):
    if spec is None or spec.p == 0.0:
        return v
    return torch.where(keep_mask(*v.shape, spec, v.device), v / (1.0 - spec.p), torch.zeros_like(v))


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * torch.special.ndtr(z),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def act_grad64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def dbl(t):
    return None if t is None else t.double()


def forward64(x, w, bias, act, spec, residual):
    """(y, z, error bound of z)."""
    z = x.double() @ w.double().t()
    M = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z = z + bias.double()
        M = M + bias.double().abs()
    bound = product_bound(x.shape[1], M, x.dtype)
    y = drop64(act64(z, act), spec)
    if residual is not None:
        y = y + residual.double()
    return y, z, bound


def check(got, want, bound, what):
    """|got - want| <= bound + one rounding to got's type, element by element."""
    tol = bound + (want.abs() + bound) * OUT_ULP[got.dtype] + 1e-42
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst error "
                           f"{(err / tol).max().item():.3g} of the bound at {bad.nonzero()[0].tolist()}")


def matrix(rows, cols, dtype, std, gen, ld=None, offset=0):
    """A [rows, cols] view with row stride ld of a buffer filled with NaN elsewhere, starting
    `offset` elements into it."""
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    v = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.copy_((torch.randn(rows, cols, generator=gen, device="cuda") * std).to(dtype))
    return v


def empty_matrix(rows, cols, dtype, ld=None, offset=0):
    """As matrix, with NaN inside too; returns (view, buffer)."""
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols], buf


def untouched(view, buf):
    """Whether every element of buf outside the view is still NaN."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool(buf[mask].isnan().all())


def workspace(rows, cin, cout, dtype, aligned=False):
    n = fs.fsdp_linear_workspace_bytes(rows, cin, cout, dtype, aligned)
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g
