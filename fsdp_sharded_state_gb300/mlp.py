"""ResidualMLP: a stack of residual MLP blocks computed between the all-gather and the
reduce-scatter of a ShardedState.

The parameters of block b are one wrap unit of the state: w1 [hidden, width], b1 [hidden],
w2 [width, hidden], b2 [width].  Forward reads them as views of the full buffer that the
all-gather fills; backward writes the weight gradients as views of a gradient replica, or
adds them to an fp32 accumulator (gradient accumulation without synchronisation), which is
what the reduce-scatter reads.  Per block, for x [rows, width]:

    h = act(x w1^T + b1);   y = x + drop(h w2^T + b2)

    gradient of y:  g = drop(dy)                         (fsdp_dropout, the forward's mask)
                    db2, dw2 = column sums of g, g^T h   (fsdp_linear_wgrad)
                    dz1 = act'(z1) * (g w2)              (fsdp_linear_dgrad)
                    db1, dw1 = column sums of dz1, dz1^T x
                    dx = dy + dz1 w1                     (fsdp_linear_dgrad, dy as the residual)

Masks are drawn from (seed, step, block, row): they are not stored, and ranks and
micro-batches that pass the index of their first row share one batch-wide mask.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import (DropoutSpec, Layout, fsdp_dropout, fsdp_linear_dgrad, fsdp_linear_forward, fsdp_linear_wgrad,
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

    def __init__(self, width: int, hidden: int, blocks: int, act: str = "gelu", p: float = 0.0, seed: int = 0):
        self.width, self.hidden, self.blocks, self.act, self.p, self.seed = width, hidden, blocks, act, p, seed
        self.saved = []
        self.stream = None         # that forward ran on

    def shapes(self):
        """(shapes, unit ids) for ShardedState: one unit per block."""
        shapes, units = [], []
        for b in range(self.blocks):
            shapes += [(self.hidden, self.width), (self.hidden,), (self.width, self.hidden), (self.width,)]
            units += [b] * 4
        return shapes, units

    def _spec(self, step: int, block: int, row0: int) -> Optional[DropoutSpec]:
        return DropoutSpec(self.p, self.seed, step * self.blocks + block, row0) if self.p else None

    def _scratch(self, x: torch.Tensor) -> torch.Tensor:
        # of one pass, on its device and, through the caching allocator, in its stream's order:
        # passes on other streams have their own.  Views of a full buffer may start at any
        # element: room for aligned copies of the operands.
        sizes = ((self.width, self.hidden), (self.hidden, self.width))           # both layers of a block
        n = max(fsdp_linear_workspace_bytes(x.shape[0], i, o, x.dtype, aligned=False) for i, o in sizes)
        return torch.empty(n, dtype=torch.uint8, device=x.device)

    def forward(self, layout: Layout, full: torch.Tensor, x: torch.Tensor, step: int = 0, row0: int = 0) -> torch.Tensor:
        """x [rows, width] through all blocks; what backward needs is kept until then."""
        v, ws = tensor_views(layout, full), self._scratch(x)
        self.saved, self.stream = [], _current_stream(x)
        for b in range(self.blocks):
            w1, b1, w2, b2 = v[4 * b:4 * b + 4]
            h = x.new_empty(x.shape[0], self.hidden)
            z = torch.empty_like(h) if self.act != "none" else None
            y = torch.empty_like(x)
            fsdp_linear_forward(x, w1, h, bias=b1, act=self.act, preact=z, workspace=ws)
            fsdp_linear_forward(h, w2, y, bias=b2, dropout=self._spec(step, b, row0), residual=x, workspace=ws)
            self.saved.append((x, z, h))
            x = y
        return x

    def backward(self, layout: Layout, full: torch.Tensor, grad: torch.Tensor, dy: torch.Tensor, step: int = 0,
                 row0: int = 0, accumulate: bool = False) -> torch.Tensor:
        """The parameters' gradients into the full-layout buffer `grad` (its dtype; added to it
        with accumulate), and the gradient of forward's x."""
        v, g, ws = tensor_views(layout, full), tensor_views(layout, grad), self._scratch(dy)
        stream = _current_stream(dy)
        for b in reversed(range(self.blocks)):
            x, z, h = self.saved.pop()
            if stream != self.stream:            # their memory is not given out again before this stream has read it
                for t in (x, z, h):
                    if t is not None:
                        t.record_stream(stream)
            w1, _, w2, _ = v[4 * b:4 * b + 4]
            gw1, gb1, gw2, gb2 = g[4 * b:4 * b + 4]
            spec = self._spec(step, b, row0)
            gy = dy
            if spec is not None:
                gy = torch.empty_like(dy)
                fsdp_dropout(dy, gy, spec)
            fsdp_linear_wgrad(gy, h, gw2, gb2, accumulate=accumulate, workspace=ws)
            dz = torch.empty_like(h)
            fsdp_linear_dgrad(gy, w2, dz, act=self.act, preact=z, workspace=ws)
            fsdp_linear_wgrad(dz, x, gw1, gb1, accumulate=accumulate, workspace=ws)
            dx = torch.empty_like(dy)
            fsdp_linear_dgrad(dz, w1, dx, residual=dy, workspace=ws)
            dy = dx
        return dy
