"""Measured cases of layer norm and of the Muon step: what a residual MLP's training step
needs beside its linear layers and AdamW.

  ln_forward    y = (x - mean) * rstd * weight + bias per row, mean and rstd kept for backward
  ln_backward   dx = residual + the gradient through the norm, and the sums over all rows that
                are the gradients of weight and bias, into a gradient replica or added to an
                fp32 accumulator
  ns            matrices brought near the closest (semi-)orthogonal one by Newton-Schulz steps
                X <- a X + b (X X^T) X + c (X X^T)^2 X from X = G / |G|
  muon          the ZeRO-1 owner step of weight matrices: mean of N gradient replicas, momentum,
                Newton-Schulz steps, decoupled weight decay, the new weights into N replicas

With `own` false, run() computes them with elementary torch operations in fp32, rounded
once at the end; with `own` true it makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}

LN_EPS = 1e-5
NS_EPS = 1e-7
NS_STEPS = 5
NS_COEFFS = (3.4445, -4.7750, 2.0315)
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _ln(name, op, rows, cols, dtype, residual=False, grad_dtype=None, accumulate=False):
    return dict(name=name, op=op, rows=rows, cols=cols, dtype=dtype, residual=residual, grad_dtype=grad_dtype or dtype,
                accumulate=accumulate)


def _ns(name, count, rows, cols, dtype):
    return dict(name=name, op="ns", count=count, rows=rows, cols=cols, dtype=dtype)


def _muon(name, blocks, width, hidden, ranks, dtype, nesterov=True):
    return dict(name=name, op="muon", blocks=blocks, width=width, hidden=hidden, ranks=ranks, dtype=dtype, nesterov=nesterov)


def listed():
    return [
        # one token's norm in front of a 2048-wide layer: the launch counts
        _ln("ln_fwd_bf16_1x2048", "ln_forward", 1, 2048, "bf16"),
        # a batch of odd length and width: rows of no 16-byte multiple
        _ln("ln_fwd_f32_333x1001", "ln_forward", 333, 1001, "f32"),
        # the residual stream of a training batch at hidden 4096
        _ln("ln_fwd_bf16_16384x4096", "ln_forward", 16384, 4096, "bf16"),
        # the tiny MLP's backward
        _ln("ln_bwd_f32_129x32", "ln_backward", 129, 32, "f32"),
        # an odd batch, the residual's gradient added
        _ln("ln_bwd_bf16_333x1001", "ln_backward", 333, 1001, "bf16", residual=True),
        # a training micro-batch at hidden 4096, weight gradients added to the fp32 accumulator
        _ln("ln_bwd_bf16_16384x4096_acc", "ln_backward", 16384, 4096, "bf16", residual=True, grad_dtype="f32", accumulate=True),
        # many short rows: the example MLP's width, the sums over the rows are the long axis
        _ln("ln_bwd_bf16_65536x256", "ln_backward", 65536, 256, "bf16", residual=True),
        # one weight of the tiny MLP: launches count
        _ns("ns_f32_64x32", 1, 64, 32, "f32"),
        # the eight equal matrices of a small stack, together
        _ns("ns_f32_8x256x1024", 8, 256, 1024, "f32"),
        # the up projection at hidden 2048 (ffn 5504)
        _ns("ns_bf16_5504x2048", 1, 5504, 2048, "bf16"),
        # a small layout of odd widths, fp32 replicas, biases between the matrices
        _muon("muon_f32_2x777x1001_N4", 2, 777, 1001, 4, "f32"),
        # a block at hidden 4096 (ffn 11008), bf16 replicas
        _muon("muon_bf16_1x4096x11008_N2", 1, 4096, 11008, 2, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 6.3e12


def _ns_flops(rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    return NS_STEPS * (m * m * n + m * m * m + 2 * m * m * n)


def draw(rng):
    op = rng.choice(["ln_forward", "ln_backward", "ln_backward", "ns", "muon"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("ln"):
        rows, cols = _log(rng, 1, 65536), _log(rng, 32, 16384)
        if rng.random() < 0.5:                   # widths of whole 16-byte rows, as most models have
            cols = max(32, cols // 32 * 32)
        rows = max(1, min(rows, 16384 * 4096 // cols))
        back = op == "ln_backward"
        grad_dtype = "f32" if back and rng.random() < 0.5 else dtype
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=back and rng.random() < 0.6, grad_dtype=grad_dtype,
                    accumulate=grad_dtype == "f32" and back and rng.random() < 0.6)
    a, b = _log(rng, 24, 4096), _log(rng, 64, 11008)
    if rng.random() < 0.5:
        a, b = max(32, a // 32 * 32), max(64, b // 64 * 64)
    if rng.random() < 0.5:
        a, b = b, a
    fit = max(1, int(MOST_FLOPS / _ns_flops(a, b)))
    if op == "ns":
        return dict(op=op, count=min(fit, rng.choice([1, 1, 2, 5, 12])), rows=a, cols=b, dtype=dtype)
    return dict(op=op, blocks=max(1, min(fit // 2, rng.choice([1, 2, 4]))), width=min(a, b), hidden=max(a, b),
                ranks=rng.choice([1, 2, 4, 8]), dtype=dtype, nesterov=rng.random() < 0.7)


def _matrices(case):
    """[(rows, cols)] of a muon case's weight matrices, in the layout's order."""
    return [(case["hidden"], case["width"]), (case["width"], case["hidden"])] * case["blocks"]


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "ns":
        R, C, n = case["rows"], case["cols"], case["count"]
        return {"bytes": 2 * n * R * C * e, "flops": n * _ns_flops(R, C)}
    if case["op"] == "muon":
        P = sum(r * c for r, c in _matrices(case))
        # gradients read, momentum and master read and written, replicas written
        state = 8 + (8 if case["dtype"] == "bf16" else 4)
        return {"bytes": P * (2 * case["ranks"] * e + state), "flops": sum(_ns_flops(r, c) for r, c in _matrices(case))}
    T, C = case["rows"], case["cols"]
    if case["op"] == "ln_forward":
        return {"bytes": 2 * T * C * e + 2 * C * e + 8 * T, "flops": 8 * T * C}
    g = SIZE[case["grad_dtype"]] * (2 if case["accumulate"] else 1)
    return {"bytes": (3 + case["residual"]) * T * C * e + C * e + 8 * T + 2 * C * g, "flops": 13 * T * C}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gradient(g, rows, cols, dt):
    """A weight gradient: noise, and about as much again in four strong directions."""
    dev = "cuda"
    u, v = (torch.randn(n, 4, generator=g, device=dev) for n in (rows, cols))
    return ((torch.randn(rows, cols, generator=g, device=dev) + 0.5 * (u @ v.t())) * 1e-3).to(dt)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "ns":
        s["src"] = [_gradient(g, case["rows"], case["cols"], dt) for _ in range(case["count"])]
        s["dst"] = [torch.empty_like(x) for x in s["src"]]
        return s
    if case["op"] == "muon":
        N, shapes = case["ranks"], []
        for r, c in _matrices(case):
            shapes += [(r, c), (r,)]                             # each weight and its bias
        P = sum(math.prod(sh) for sh in shapes)
        full = torch.randn(P, generator=g, device=dev) * 0.02    # the parameters, tensors back to back
        s["shapes"], s["params"] = shapes, [full.to(dt) for _ in range(N)]
        s["grads"], at = [torch.empty(P, dtype=dt, device=dev) for _ in range(N)], 0
        s["master"], s["momentum"], s["at"] = [], [], []
        for sh in shapes:
            n = math.prod(sh)
            if len(sh) == 2:
                for q in range(N):
                    s["grads"][q][at:at + n] = _gradient(g, sh[0], sh[1], dt).reshape(-1)
                s["at"].append((at, n))
                s["master"].append(full[at:at + n].view(sh).clone() if dt != torch.float32 else None)
                s["momentum"].append(torch.randn(sh, generator=g, device=dev) * 1e-3)
            else:
                for q in range(N):
                    s["grads"][q][at:at + n] = (torch.randn(n, generator=g, device=dev) * 1e-3).to(dt)
            at += n
        return s
    T, C, gdt = case["rows"], case["cols"], DTYPES[case["grad_dtype"]]

    def rnd(rows, std, dtype=dt):
        return (torch.randn(rows, C, generator=g, device=dev) * std).to(dtype)

    # a residual stream: every column with an offset of its own
    s["x"] = (torch.randn(T, C, generator=g, device=dev) * 1.5 + torch.randn(1, C, generator=g, device=dev) * 0.5).to(dt)
    s["weight"], s["bias"] = (1.0 + rnd(1, 0.1).float()).to(dt).reshape(-1), rnd(1, 0.1).reshape(-1)
    if case["op"] == "ln_forward":
        s["y"] = torch.empty(T, C, dtype=dt, device=dev)
        s["mean"], s["rstd"] = torch.empty(T, device=dev), torch.empty(T, device=dev)
        return s
    x = s["x"].double()
    s["mean"], s["rstd"] = x.mean(1).float(), ((x.var(1, unbiased=False) + LN_EPS) ** -0.5).float()
    s["dy"] = rnd(T, 1e-3)
    s["residual"] = rnd(T, 1e-3) if case["residual"] else None
    s["dx"] = torch.empty(T, C, dtype=dt, device=dev)
    s["dw"], s["db"] = rnd(1, 1e-3, gdt).reshape(-1), rnd(1, 1e-3, gdt).reshape(-1)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _newton_schulz(g):
    x = g.float()
    x = x / torch.clamp_min(x.square().sum().sqrt(), NS_EPS)
    a, b, c = NS_COEFFS
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    for _ in range(NS_STEPS):
        gram = x @ x.t()
        poly = b * gram + c * (gram @ gram)
        x = a * x + poly @ x
    return x.t() if tall else x


def _scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


def _plain_muon(s):
    case = s["case"]
    for i, (at, n) in enumerate(s["at"]):
        m = s["momentum"][i]
        grad = s["grads"][0][at:at + n].float()
        for q in range(1, case["ranks"]):
            grad = grad + s["grads"][q][at:at + n].float()
        grad = (grad / case["ranks"]).view(m.shape)
        m.copy_(MOMENTUM * m + (1.0 - MOMENTUM) * grad)
        u = (1.0 - MOMENTUM) * grad + MOMENTUM * m if case["nesterov"] else m
        w = s["master"][i] if s["master"][i] is not None else s["params"][0][at:at + n].view(m.shape)
        w = (1.0 - LR * DECAY) * w - LR * _scale(*m.shape) * _newton_schulz(u)
        if s["master"][i] is not None:
            s["master"][i].copy_(w)
        for p in s["params"]:
            p[at:at + n] = w.reshape(-1).to(p.dtype)
    return _muon_outputs(s)


def _muon_outputs(s):
    out = {"params": s["params"], "momentum": s["momentum"]}
    if s["case"]["dtype"] == "bf16":
        out["master"] = s["master"]
    return out


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "ns":
        return [_newton_schulz(x).to(dt) for x in s["src"]]
    if op == "muon":
        return _plain_muon(s)
    x, w = s["x"].float(), s["weight"].float()
    if op == "ln_forward":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + LN_EPS)
        return {"y": (d * rstd * w + s["bias"].float()).to(dt), "mean": mean.reshape(-1), "rstd": rstd.reshape(-1)}
    dy, rstd = s["dy"].float(), s["rstd"].reshape(-1, 1)
    xhat = (x - s["mean"].reshape(-1, 1)) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    if case["accumulate"]:
        s["dw"] += dw
        s["db"] += db
    else:
        s["dw"].copy_(dw)
        s["db"].copy_(db)
    return {"dx": dx.to(dt), "dw": s["dw"], "db": s["db"]}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import fsdp_sharded_state_gb300 as fs
    case = s["case"]
    op = case["op"]
    if op == "ln_forward":
        fs.fsdp_layernorm_forward(s["x"], s["y"], weight=s["weight"], bias=s["bias"], mean=s["mean"], rstd=s["rstd"], eps=LN_EPS)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_backward":
        if "workspace" not in s:                 # scratch, kept as a program keeps it
            n = fs.fsdp_layernorm_workspace_bytes(case["rows"], case["cols"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        fs.fsdp_layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], weight=s["weight"], dw=s["dw"], db=s["db"],
                                   residual=s["residual"], accumulate=case["accumulate"], workspace=s["workspace"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "ns":
        if "workspace" not in s:
            n = fs.fsdp_newton_schulz_workspace_bytes(case["count"], case["rows"], case["cols"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        fs.fsdp_newton_schulz(s["src"], s["dst"], steps=NS_STEPS, eps=NS_EPS, workspace=s["workspace"])
        return s["dst"]
    if "layout" not in s:                        # the owner rows of the sharded optimizer state, filled once
        s["layout"] = L = fs.Layout(s["shapes"], n_ranks=case["ranks"], mode=fs.FSDP_ZERO1)
        s["tensors"] = [t for t, sh in enumerate(s["shapes"]) if len(sh) == 2]
        rows = {}
        for name in ("momentum", "master"):
            if s[name][0] is None:
                rows[name] = None
                continue
            rows[name] = torch.zeros(L.N, L.stride, device="cuda")
            for i, t in enumerate(s["tensors"]):
                at, old = L.tensor(t)["shard_off"], s[name][i]
                v = rows[name][L.owner(t), at:at + old.numel()].view(old.shape)
                v.copy_(old)
                s[name][i] = v                   # the outputs are views of the rows
        s["rows"] = rows
        s["hp"] = fs.MuonHparams(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, eps=NS_EPS, nesterov=case["nesterov"],
                                 steps=NS_STEPS, scale="rms")
        n = fs.fsdp_zero1_muon_workspace_bytes(L, s["tensors"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    fs.fsdp_zero1_muon_broadcast(s["layout"], s["tensors"], s["grads"], s["rows"]["master"], s["rows"]["momentum"], s["params"],
                                 s["hp"], workspace=s["workspace"])
    return _muon_outputs(s)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_orthogonal(g):
    """U p(S) V^T, p the steps' odd polynomial, from the eigenvectors of the smaller Gram matrix."""
    tall = g.shape[0] > g.shape[1]
    x = (g.T if tall else g) / max(float(torch.linalg.matrix_norm(g)), NS_EPS)
    lam, vec = torch.linalg.eigh(torch.mm(x, x.T))
    t, gain = lam.clamp(min=0.0), torch.ones_like(lam)           # squared singular values; what each was multiplied by
    for _ in range(NS_STEPS):
        q = NS_COEFFS[0] + t * (NS_COEFFS[1] + t * NS_COEFFS[2])
        gain, t = gain * q, t * q * q
    o = torch.mm(vec * gain, torch.mm(vec.T, x))
    return o.T if tall else o


def exact(case, seed):
    s = prepare(case, seed)
    D = lambda t: t.to(torch.float64)
    if case["op"] == "ns":
        return [_exact_orthogonal(D(x)) for x in s["src"]]
    if case["op"] == "muon":
        params, mom, mas = [D(p) for p in s["params"]], [], []
        for (at, n), m, w in zip(s["at"], s["momentum"], s["master"]):
            part = slice(at, at + n)
            g = torch.stack([D(r[part]) for r in s["grads"]]).mean(0).view(m.shape)
            mom.append(torch.lerp(g, D(m), MOMENTUM))
            u = torch.lerp(g, mom[-1], MOMENTUM) if case["nesterov"] else mom[-1]
            w = D(s["params"][0][part]).view(m.shape) if w is None else D(w)
            mas.append(w * (1 - LR * DECAY) - LR * 0.2 * max(m.shape) ** 0.5 * _exact_orthogonal(u))
            for p in params:
                p[part] = mas[-1].reshape(-1)
        out = {"params": params, "momentum": mom}
        if case["dtype"] == "bf16":
            out["master"] = mas
        return out
    x = D(s["x"])
    if case["op"] == "ln_forward":
        var, mean = torch.var_mean(x, 1, correction=0)
        y = torch.nn.functional.layer_norm(x, (x.shape[1],), D(s["weight"]), D(s["bias"]), LN_EPS)
        return {"y": y, "mean": mean, "rstd": torch.rsqrt(var + LN_EPS)}
    n, dy, w, r = case["cols"], D(s["dy"]), D(s["weight"]), D(s["rstd"])
    h = torch.einsum("tc,t->tc", x - D(s["mean"])[:, None], r)
    p, q = torch.einsum("tc,c->t", dy, w) / n, torch.einsum("tc,c,tc->t", dy, w, h) / n
    dx = r[:, None] * (dy * w - p[:, None] - q[:, None] * h)
    if s["residual"] is not None:
        dx += D(s["residual"])
    dw, db = torch.einsum("tc,tc->c", dy, h), torch.einsum("tc->c", dy)
    if case["accumulate"]:
        dw, db = dw + D(s["dw"]), db + D(s["db"])
    return {"dx": dx, "dw": dw, "db": db}
