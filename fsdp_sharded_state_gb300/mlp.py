"""ResidualMLP: a stack of residual MLP blocks computed between the all-gather and the
reduce-scatter of a ShardedState.

The parameters of block b are one wrap unit of the state: w1 [hidden, width], b1 [hidden],
w2 [width, hidden], b2 [width], and, with norm, the weight and bias g, c [width] of the layer norm
in front of them.  Forward reads them as views of the full buffer that the
all-gather fills; backward writes the weight gradients as views of a gradient replica, or
adds them to an fp32 accumulator (gradient accumulation without synchronisation), which is
what the reduce-scatter reads.  Per block, for x [rows, width]:

    n = norm(x) g + c, or x itself                       (fsdp_layernorm_forward)
    h = act(n w1^T + b1);   y = x + drop(h w2^T + b2)

    gradient of y:  e = drop(dy)                         (fsdp_dropout, the forward's mask)
                    db2, dw2 = column sums of e, e^T h   (fsdp_linear_wgrad)
                    dz1 = act'(z1) * (e w2)              (fsdp_linear_dgrad)
                    db1, dw1 = column sums of dz1, dz1^T n
                    dx = dy + dz1 w1                     (fsdp_linear_dgrad, dy as the residual)
    or, with norm,  dn = dz1 w1;  dx = dy + the norm's gradient of dn, with those of g and c
                                                         (fsdp_layernorm_backward, dy as the residual)

Masks are drawn from (seed, step, block, row): they are not stored, and ranks and
micro-batches that pass the index of their first row share one batch-wide mask.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import (DropoutSpec, Layout, fsdp_dropout, fsdp_layernorm_backward, fsdp_layernorm_forward,
               fsdp_layernorm_workspace_bytes, fsdp_linear_dgrad, fsdp_linear_forward, fsdp_linear_wgrad,
               fsdp_linear_workspace_bytes)


def tensor_views(layout: Layout, full: torch.Tensor) -> List[torch.Tensor]:
    """The layout's tensors as views of a full-layout buffer (parameters or gradients)."""
    out = []
    for t, shape in enumerate(layout.shapes):
        d = layout.tensor(t)
        out.append(full[d["full_off"]:d["full_off"] + d["numel"]].view(shape))
    return out


def _current_stream(t: torch.Tensor):
    return torch.cuda.current_stream(t.device) if t.is_cuda else None


class ResidualMLP:
    """Forward and backward of `blocks` residual MLP blocks over full-layout buffers."""

    def __init__(self, width: int, hidden: int, blocks: int, act: str = "gelu", p: float = 0.0, seed: int = 0,
                 norm: bool = False, eps: float = 1e-5):
        self.width, self.hidden, self.blocks, self.act, self.p, self.seed = width, hidden, blocks, act, p, seed
        self.norm, self.eps = norm, eps
        self.per_block = 6 if norm else 4          # tensors
        self.saved = []
        self.stream = None         # that forward ran on

    def shapes(self):
        """(shapes, unit ids) for ShardedState: one unit per block."""
        shapes, units = [], []
        for b in range(self.blocks):
            shapes += [(self.hidden, self.width), (self.hidden,), (self.width, self.hidden), (self.width,)]
            shapes += [(self.width,), (self.width,)] if self.norm else []
            units += [b] * self.per_block
        return shapes, units

    def initialise(self, layout: Layout, full: torch.Tensor, generator=None) -> None:
        """Weights ~ N(0, 1 / fan-in), biases 0, the norms' weights 1, into a full-layout buffer."""
        for t, v in enumerate(tensor_views(layout, full)):
            if v.dim() == 2:
                v.copy_(torch.randn(v.shape, generator=generator, device=v.device) * v.shape[1] ** -0.5)
            else:
                v.fill_(1.0 if t % self.per_block == 4 else 0.0)

    def _spec(self, step: int, block: int, row0: int) -> Optional[DropoutSpec]:
        return DropoutSpec(self.p, self.seed, step * self.blocks + block, row0) if self.p else None

    def _scratch(self, x: torch.Tensor) -> torch.Tensor:
        # of one pass, on its device and, through the caching allocator, in its stream's order:
        # passes on other streams have their own.  Views of a full buffer may start at any
        # element: room for aligned copies of the operands.
        sizes = ((self.width, self.hidden), (self.hidden, self.width))           # both layers of a block
        n = max(fsdp_linear_workspace_bytes(x.shape[0], i, o, x.dtype, aligned=False) for i, o in sizes)
        if self.norm:
            n = max(n, fsdp_layernorm_workspace_bytes(x.shape[0], self.width))
        return torch.empty(n, dtype=torch.uint8, device=x.device)

    def forward(self, layout: Layout, full: torch.Tensor, x: torch.Tensor, step: int = 0, row0: int = 0) -> torch.Tensor:
        """x [rows, width] through all blocks; what backward needs is kept until then."""
        v, ws = tensor_views(layout, full), self._scratch(x)
        self.saved, self.stream = [], _current_stream(x)
        for b in range(self.blocks):
            w1, b1, w2, b2, *nv = v[self.per_block * b:self.per_block * (b + 1)]
            h = x.new_empty(x.shape[0], self.hidden)
            z = torch.empty_like(h) if self.act != "none" else None
            y = torch.empty_like(x)
            n, kept = x, ()
            if self.norm:
                n = torch.empty_like(x)
                mean, rstd = (torch.empty(x.shape[0], dtype=torch.float32, device=x.device) for _ in range(2))
                fsdp_layernorm_forward(x, n, nv[0], nv[1], mean, rstd, self.eps)
                kept = (n, mean, rstd)
            fsdp_linear_forward(n, w1, h, bias=b1, act=self.act, preact=z, workspace=ws)
            fsdp_linear_forward(h, w2, y, bias=b2, dropout=self._spec(step, b, row0), residual=x, workspace=ws)
            self.saved.append((x, z, h) + kept)
            x = y
        return x

    def backward(self, layout: Layout, full: torch.Tensor, grad: torch.Tensor, dy: torch.Tensor, step: int = 0,
                 row0: int = 0, accumulate: bool = False) -> torch.Tensor:
        """The parameters' gradients into the full-layout buffer `grad` (its dtype; added to it
        with accumulate), and the gradient of forward's x."""
        v, g, ws = tensor_views(layout, full), tensor_views(layout, grad), self._scratch(dy)
        stream = _current_stream(dy)
        for b in reversed(range(self.blocks)):
            saved = self.saved.pop()
            if stream != self.stream:            # their memory is not given out again before this stream has read it
                for t in saved:
                    if t is not None:
                        t.record_stream(stream)
            x, z, h, *kept = saved
            w1, _, w2, _, *nv = v[self.per_block * b:self.per_block * (b + 1)]
            gw1, gb1, gw2, gb2, *gn = g[self.per_block * b:self.per_block * (b + 1)]
            spec = self._spec(step, b, row0)
            gy = dy
            if spec is not None:
                gy = torch.empty_like(dy)
                fsdp_dropout(dy, gy, spec)
            fsdp_linear_wgrad(gy, h, gw2, gb2, accumulate=accumulate, workspace=ws)
            dz = torch.empty_like(h)
            fsdp_linear_dgrad(gy, w2, dz, act=self.act, preact=z, workspace=ws)
            fsdp_linear_wgrad(dz, kept[0] if kept else x, gw1, gb1, accumulate=accumulate, workspace=ws)
            dx = torch.empty_like(dy)
            if kept:
                _, mean, rstd = kept
                fsdp_linear_dgrad(dz, w1, dx, workspace=ws)
                fsdp_layernorm_backward(dx, x, mean, rstd, dx, nv[0], gn[0], gn[1], residual=dy, accumulate=accumulate, workspace=ws)
            else:
                fsdp_linear_dgrad(dz, w1, dx, residual=dy, workspace=ws)
            dy = dx
        return dy
