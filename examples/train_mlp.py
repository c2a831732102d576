#!/usr/bin/env python
"""Trains a residual MLP on a synthetic regression task with the sharded state of N
simulated data-parallel ranks: per step one all-gather, forward and backward of every
rank's batch on the full buffer, then the fused reduce-scatter + AdamW + cast.

  python examples/train_mlp.py [--width 256] [--hidden 1024] [--blocks 2] [--ranks 4]
                               [--rows 512] [--micro 1] [--steps 30] [--p 0.1] [--dtype bf16]

--micro k splits every rank's rows into k micro-batches whose gradients add up in fp32
accumulators (no synchronisation before the last one).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fsdp_sharded_state_gb300 as fs  # noqa: E402


def initial_parameters(layout, dtype, device, seed=0):
    """Weights ~ N(0, 1 / fan-in), biases 0, as a full-layout buffer."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    full = torch.zeros(layout.info["full_numel"], dtype=torch.float32, device=device)
    for v in fs.tensor_views(layout, full):
        if v.dim() == 2:
            v.copy_(torch.randn(v.shape, generator=g, device=device) * v.shape[1] ** -0.5)
    return full.to(dtype)


def train(width=256, hidden=1024, blocks=2, ranks=4, rows=512, micro=1, steps=30, p=0.1, dtype=torch.bfloat16,
          lr=1e-3, device="cuda", say=print):
    mlp = fs.ResidualMLP(width, hidden, blocks, act="gelu", p=p, seed=1234)
    shapes, units = mlp.shapes()
    st = fs.ShardedState(shapes, units, ranks, param_dtype=dtype, device=device)
    st.init_from_full(initial_parameters(st.layout, dtype, device))
    # fp32 gradient replicas: with micro-batches, the accumulators
    grads = [torch.zeros(st.F, dtype=torch.float32, device=device) for _ in range(ranks)]
    g = torch.Generator(device=device)
    g.manual_seed(7)
    teacher = torch.randn(width, width, generator=g, device=device) * width ** -0.5
    hp = (lr, 0.9, 0.999, 1e-8, 0.0)
    losses = []
    for step in range(steps):
        st.unshard()
        loss = torch.zeros((), device=device)
        for r in range(ranks):
            for m in range(micro):
                n = rows // micro
                x = torch.randn(n, width, generator=g, device=device)
                target = x + torch.tanh(x @ teacher)
                row0 = (r * micro + m) * n                  # of the batch over all ranks
                y = mlp.forward(st.layout, st.full, x.to(dtype), step, row0)
                diff = y.float() - target
                loss += diff.square().mean() / (ranks * micro)
                dy = (diff * (2.0 / (diff.numel() * micro))).to(dtype)
                mlp.backward(st.layout, st.full, grads[r], dy, step, row0, accumulate=m > 0)
        st.reduce_scatter_adamw(grads, hp)
        losses.append(float(loss))
        if step % 5 == 0 or step == steps - 1:
            say(f"step {step:3d}  loss {losses[-1]:.4f}")
    fs.fsdp_check_status()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("width", 256), ("hidden", 1024), ("blocks", 2), ("ranks", 4), ("rows", 512), ("micro", 1),
                          ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--p", type=float, default=0.1)
    ap.add_argument("--lr", type=float, default=1e-3)
    ap.add_argument("--dtype", choices=("bf16", "fp32"), default="bf16")
    a = ap.parse_args()
    train(a.width, a.hidden, a.blocks, a.ranks, a.rows, a.micro, a.steps, a.p,
          torch.bfloat16 if a.dtype == "bf16" else torch.float32, a.lr)


if __name__ == "__main__":
    main()
