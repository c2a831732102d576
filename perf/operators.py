"""Measured cases of the layer operators: linear layers and dropout, forward and backward.

A training loop around the sharded-state step computes its layers between the all-gather
that fills the full parameter buffer and the reduce-scatter that reads the gradient
replicas.  The operators measured here are that part:

  forward   y = residual + dropout(act(x w^T + bias)), the pre-activation kept for backward
  dgrad     dx = residual + act'(z) * dropout(dz w), the gradient for the layer before
  wgrad     dw (+)= dz^T x and db (+)= column sums of dz, into a gradient replica or an
            fp32 accumulator
  dropout   y = residual + keep * x / (1 - p) with keep drawn from a counter-based
            generator, the same call forward and backward

With `own` false, run() computes them with elementary torch operations in fp32, rounded
once at the end; with `own` true it makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, rows, cols_in, cols_out, dtype, **opt):
    c = dict(name=name, op=op, rows=rows, cols_in=cols_in, cols_out=cols_out, dtype=dtype, act="none", bias=False,
             p=0.0, residual=False, grad_dtype=dtype, accumulate=False)
    c.update(opt)
    return c


def listed():
    return [
        # one token through a 2048-wide layer: the launch and one read of the weight count
        _case("fwd_bf16_1x2048x2048", "forward", 1, 2048, 2048, "bf16", act="gelu", bias=True),
        # a batch of odd length through odd widths: rows of no 16-byte multiple
        _case("fwd_bf16_333x1001x777", "forward", 333, 1001, 777, "bf16", act="silu", bias=True, residual=True, p=0.1),
        # the 128 MiB MLP's fp32 layer on a ragged batch
        _case("fwd_f32_1000x2048x2048", "forward", 1000, 2048, 2048, "f32", act="relu", bias=True),
        # the down projection of a block at hidden 4096: dropout and the residual stream in the epilogue
        _case("fwd_bf16_8192x11008x4096", "forward", 8192, 11008, 4096, "bf16", bias=True, residual=True, p=0.1),
        # the output projection onto 32000 columns, the largest weight of the layouts
        _case("fwd_bf16_8192x4096x32000", "forward", 8192, 4096, 32000, "bf16"),
        # the tiny MLP backward, fp32
        _case("dgrad_f32_129x32x64", "dgrad", 129, 32, 64, "f32", act="relu"),
        # gradient through the up projection's activation at hidden 2048 (ffn 5504)
        _case("dgrad_bf16_4096x5504x2048", "dgrad", 4096, 5504, 2048, "bf16", act="gelu", p=0.1),
        # weight gradient of the down projection into a bf16 gradient replica
        _case("wgrad_bf16_8192x11008x4096", "wgrad", 8192, 11008, 4096, "bf16", bias=True),
        # a micro-batch added to the fp32 accumulator of a 2048-wide layer
        _case("wgrad_bf16_2048x2048x2048_acc", "wgrad", 2048, 2048, 2048, "bf16", bias=True, grad_dtype="f32", accumulate=True),
        # many rows, a small fp32 layer: the sum over the rows is the long axis
        _case("wgrad_f32_16384x64x32", "wgrad", 16384, 64, 32, "f32", bias=True),
        # dropout of one short ragged fp32 batch, and of the residual stream at hidden 4096
        _case("dropout_f32_77x1001", "dropout", 77, 1001, 1001, "f32", p=0.5),
        _case("dropout_bf16_16384x4096", "dropout", 16384, 4096, 4096, "bf16", p=0.1, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "dgrad", "dgrad", "wgrad", "wgrad", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows, ci, co = _log(rng, 1, 16384), _log(rng, 32, 11008), _log(rng, 32, 11008)
    if rng.random() < 0.5:                       # widths of whole 16-byte rows, as most models have
        ci, co = max(32, ci // 32 * 32), max(32, co // 32 * 32)
    # at most 16384 x 11008 x 11008: 4 TFLOP, twice the largest listed case; cut the rows to stay under it
    if op != "dropout":
        rows = min(rows, 8192 * 4096 * 32000 // (ci * co))
    c = dict(op=op, rows=rows, cols_in=ci, cols_out=ci if op == "dropout" else co, dtype=dtype,
             act=rng.choice(["none", "relu", "gelu", "silu"]) if op in ("forward", "dgrad") else "none",
             bias=op in ("forward", "wgrad") and rng.random() < 0.7,
             p=rng.choice([0.1, 0.2, 0.5]) if op == "dropout" or (op != "wgrad" and rng.random() < 0.4) else 0.0,
             residual=op != "wgrad" and rng.random() < 0.4, grad_dtype=dtype, accumulate=False)
    if op == "wgrad":
        c["grad_dtype"] = "f32" if rng.random() < 0.5 else dtype
        c["accumulate"] = c["grad_dtype"] == "f32" and rng.random() < 0.5
    return c


def work(case):
    T, I, O, e = case["rows"], case["cols_in"], case["cols_out"], SIZE[case["dtype"]]
    res = case["residual"]
    if case["op"] == "dropout":
        return {"bytes": (2 + res) * T * I * e, "flops": T * I * (2 + res)}
    if case["op"] == "forward":
        keep = case["act"] != "none"             # the pre-activation is written too
        return {"bytes": (T * I + O * I + T * O * (1 + res + keep) + (O if case["bias"] else 0)) * e, "flops": 2 * T * I * O}
    if case["op"] == "dgrad":
        z = case["act"] != "none"
        return {"bytes": (T * O + O * I + T * I * (1 + res + z)) * e, "flops": 2 * T * I * O}
    g = SIZE[case["grad_dtype"]] * (2 if case["accumulate"] else 1)
    return {"bytes": T * (I + O) * e + O * I * g + (O * g if case["bias"] else 0), "flops": 2 * T * I * O}


# ---------------------------------------------------------------------------
# inputs: activations ~ N(0, 1), weights ~ N(0, 0.02), gradients ~ N(0, 1e-3)
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, I, O = case["rows"], case["cols_in"], case["cols_out"]

    def rnd(rows, cols, std, dtype=dt):
        return (torch.randn(rows, cols, generator=g, device=dev) * std).to(dtype)

    s = {"case": case, "seed": seed * 2654435761 % (1 << 62) + 12345, "layer": 3}
    op = case["op"]
    if op == "dropout":
        s["x"] = rnd(T, I, 1.0)
        s["residual"] = rnd(T, I, 1.0) if case["residual"] else None
        s["y"] = torch.empty(T, I, dtype=dt, device=dev)
    elif op == "forward":
        s["x"], s["w"] = rnd(T, I, 1.0), rnd(O, I, 0.02)
        s["bias"] = rnd(1, O, 0.02).reshape(-1) if case["bias"] else None
        s["residual"] = rnd(T, O, 1.0) if case["residual"] else None
        s["y"] = torch.empty(T, O, dtype=dt, device=dev)
        s["preact"] = torch.empty(T, O, dtype=dt, device=dev) if case["act"] != "none" else None
    elif op == "dgrad":
        s["dz"], s["w"] = rnd(T, O, 1e-3), rnd(O, I, 0.02)
        s["preact"] = rnd(T, I, 1.0) if case["act"] != "none" else None
        s["residual"] = rnd(T, I, 1e-3) if case["residual"] else None
        s["dx"] = torch.empty(T, I, dtype=dt, device=dev)
    else:
        gdt = DTYPES[case["grad_dtype"]]
        s["dz"], s["x"] = rnd(T, O, 1e-3), rnd(T, I, 1.0)
        s["dw"], s["db"] = rnd(O, I, 1e-3, gdt), rnd(1, O, 1e-3, gdt).reshape(-1) if case["bias"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
M32 = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011) on int64 tensors holding 32-bit words."""
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57          # exact modulo 2^64
        c0, c1, c2, c3 = ((p1 >> 32) & M32) ^ c1 ^ k0, p1 & M32, ((p0 >> 32) & M32) ^ c3 ^ k1, p0 & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return c0, c1, c2, c3


def _keep(state, rows, cols):
    """keep[r, c]: word c % 4 of Philox(counter = (c / 4, r, 0, layer), key = seed) >= p * 2^32."""
    dev = "cuda"
    q = torch.arange((cols + 3) // 4, device=dev, dtype=torch.int64).reshape(1, -1)
    r = torch.arange(rows, device=dev, dtype=torch.int64).reshape(-1, 1)
    zero = torch.zeros(rows, q.shape[1], device=dev, dtype=torch.int64)
    seed = state["seed"]
    words = _philox(zero + q, zero + r, zero, zero + state["layer"], seed & M32, seed >> 32)
    return torch.stack(words, -1).reshape(rows, -1)[:, :cols] >= int(state["case"]["p"] * 4294967296.0)


def _drop(state, v):
    p = state["case"]["p"]
    if p == 0.0:
        return v
    return torch.where(_keep(state, *v.shape), v * (1.0 / (1.0 - p)), torch.zeros((), device=v.device))


def _act(z, kind):
    if kind == "relu":
        return torch.clamp_min(z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "dropout":
        y = _drop(s, s["x"].float())
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt)}
    if op == "forward":
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _drop(s, _act(z, case["act"]))
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "preact": z.to(dt)} if case["act"] != "none" else {"y": y.to(dt)}
    if op == "dgrad":
        g = _drop(s, s["dz"].float() @ s["w"].float())
        if case["act"] != "none":
            g = g * _act_grad(s["preact"].float(), case["act"])
        if s["residual"] is not None:
            g = g + s["residual"].float()
        return {"dx": g.to(dt)}
    dz = s["dz"].float()
    dw, db = dz.t() @ s["x"].float(), dz.sum(0) if s["db"] is not None else None
    if case["accumulate"]:
        s["dw"] += dw
        if db is not None:
            s["db"] += db
    else:
        s["dw"].copy_(dw)
        if db is not None:
            s["db"].copy_(db)
    return {"dw": s["dw"], "db": s["db"]}


def _own(s):
    import fsdp_sharded_state_gb300 as fs
    case = s["case"]
    op = case["op"]
    drop = fs.DropoutSpec(case["p"], s["seed"], s["layer"]) if case["p"] else None
    if op == "dropout":
        fs.fsdp_dropout(s["x"], s["y"], drop, residual=s["residual"])
        return {"y": s["y"]}
    if "workspace" not in s:                     # scratch of the three linear calls, kept as a program keeps it
        n = fs.fsdp_linear_workspace_bytes(case["rows"], case["cols_in"], case["cols_out"], DTYPES[case["dtype"]])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    if op == "forward":
        fs.fsdp_linear_forward(s["x"], s["w"], s["y"], bias=s["bias"], act=case["act"], preact=s["preact"], dropout=drop,
                               residual=s["residual"], workspace=s["workspace"])
        return {"y": s["y"], "preact": s["preact"]} if case["act"] != "none" else {"y": s["y"]}
    if op == "dgrad":
        fs.fsdp_linear_dgrad(s["dz"], s["w"], s["dx"], act=case["act"], preact=s["preact"], dropout=drop,
                             residual=s["residual"], workspace=s["workspace"])
        return {"dx": s["dx"]}
    fs.fsdp_linear_wgrad(s["dz"], s["x"], s["dw"], s["db"], accumulate=case["accumulate"], workspace=s["workspace"])
    return {"dw": s["dw"], "db": s["db"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_keep(seed, layer, rows, cols, p):
    """The kept positions, drawn with numpy's unsigned integers."""
    nq = -(-cols // 4)
    c = [np.tile(np.arange(nq, dtype=np.uint64), rows), np.repeat(np.arange(rows, dtype=np.uint64), nq),
         np.zeros(rows * nq, np.uint64), np.full(rows * nq, layer, np.uint64)]
    lo, k = np.uint64(M32), [seed & M32, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & lo, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    keep = np.stack(c, -1).reshape(rows, 4 * nq)[:, :cols] >= np.uint64(math.floor(p * 2.0 ** 32))
    return torch.from_numpy(keep).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op, p, kind = case["op"], case["p"], case["act"]
    D = lambda t: t.to(torch.float64)

    def dropped(v):
        return v if p == 0.0 else D(_exact_keep(s["seed"], s["layer"], v.shape[0], v.shape[1], p)) * v / (1.0 - p)

    def plus_residual(v):
        return v if s["residual"] is None else v + D(s["residual"])

    if op == "dropout":
        return {"y": plus_residual(dropped(D(s["x"])))}
    if op == "forward":
        z = torch.mm(D(s["x"]), D(s["w"]).T)
        if s["bias"] is not None:
            z += D(s["bias"])[None, :]
        a = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0 * z),
             "gelu": lambda: z * torch.special.ndtr(z), "silu": lambda: z * torch.sigmoid(z)}[kind]()
        y = plus_residual(dropped(a))
        return {"y": y} if kind == "none" else {"y": y, "preact": z}
    if op == "dgrad":
        gx = dropped(torch.mm(D(s["dz"]), D(s["w"])))
        if kind != "none":
            z = D(s["preact"]).requires_grad_()
            a = {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[kind](z)
            gx = torch.autograd.grad(a, z, gx)[0]
        return {"dx": plus_residual(gx)}
    dw, db = torch.mm(D(s["dz"]).T, D(s["x"])), D(s["dz"]).sum(dim=0)
    if case["accumulate"]:
        dw, db = D(s["dw"]) + dw, db if s["db"] is None else D(s["db"]) + db
    return {"dw": dw, "db": db if s["db"] is not None else None}
