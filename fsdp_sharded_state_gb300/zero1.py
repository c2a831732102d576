"""Zero1State: the buffers of a ZeRO-1 training state and its step, with Muon for the weight matrices
and AdamW for the rest ("NCCL ZeRO/FSDP state sharding", section "ZeRO-1：Optimizer State Sharding").

Parameters are whole on every one of the N simulated ranks; each tensor's momentum, second moment
and master copy live on its owner rank alone.  A step reduces the N gradient replicas, updates every
tensor at its owner and writes the new parameters into all N replicas.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import (FSDP_BF16, FSDP_F32, FSDP_ZERO1, Layout, MuonHparams, fsdp_reshard, fsdp_zero1_adamw_broadcast,
               fsdp_zero1_muon_broadcast, fsdp_zero1_muon_workspace_bytes)
from .state import as_stream, whole_on_stream


class Zero1State:
    def __init__(self, shapes: Sequence[Sequence[int]], n_ranks: int, param_dtype: torch.dtype = torch.bfloat16,
                 muon: Optional[Sequence[int]] = None, device="cuda"):
        """muon: indices of the tensors that Muon updates; by default those of two dimensions and more
        than one column.  Neighbouring tensors of one optimizer make a unit of the layout."""
        if param_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("param_dtype must be bfloat16 or float32")
        shapes = [tuple(s) for s in shapes]
        self.muon = [t for t, s in enumerate(shapes) if len(s) == 2 and s[0] > 0 and s[1] > 1] if muon is None else list(muon)
        kind = [t in set(self.muon) for t in range(len(shapes))]
        units = [0] * len(shapes)
        for t in range(1, len(shapes)):
            units[t] = units[t - 1] + (kind[t] != kind[t - 1])
        self.adamw_units = sorted({u for u, k in zip(units, kind) if not k})
        code = FSDP_BF16 if param_dtype == torch.bfloat16 else FSDP_F32
        self.layout = Layout(shapes, units, n_ranks, FSDP_ZERO1, [code] * len(shapes))
        self.N, dev = n_ranks, torch.device(device)
        rows = lambda: torch.zeros(self.N, self.layout.stride, dtype=torch.float32, device=dev)
        self.master = rows() if param_dtype == torch.bfloat16 else None
        self.exp_avg, self.exp_avg_sq = rows(), rows()       # Muon's momentum is its tensors' part of exp_avg
        self.params = [torch.zeros(self.layout.info["full_numel"], dtype=param_dtype, device=dev) for _ in range(self.N)]
        self.t = 0

    def init_from_full(self, full: torch.Tensor, stream=None) -> None:
        """Parameters of a constructed model (fp32 or bf16, full layout) into all replicas and the
        master rows; moments to zero.  All of it on `stream` (the current one by default), after what
        the current stream held before the call and before what it is given next."""
        with whole_on_stream(stream, self.exp_avg.device):
            if self.master is not None:
                fsdp_reshard(self.layout, 0, self.layout.n_units, full, self.master, None, stream)
            for p in self.params:
                p.copy_(full)
            self.exp_avg.zero_()
            self.exp_avg_sq.zero_()
        self.t = 0

    def step(self, grads, muon: Optional[MuonHparams] = None, adamw=(1e-3, 0.9, 0.999, 1e-8, 0.01), workspace=None,
             stream=None) -> None:
        """One step from N gradient replicas.  workspace: fsdp_zero1_muon_workspace_bytes of the layout and
        self.muon; by default of the call's own, from the caching allocator on the call's stream."""
        t = self.t + 1
        if self.muon:
            if workspace is None:
                n, dev = fsdp_zero1_muon_workspace_bytes(self.layout, self.muon), self.exp_avg.device
                # that stream's own memory: other streams' may still be in use there, or be given away too soon
                with torch.cuda.stream(as_stream(stream, dev)):
                    workspace = torch.empty(n, dtype=torch.uint8, device=dev)
            fsdp_zero1_muon_broadcast(self.layout, self.muon, grads, self.master, self.exp_avg, self.params, muon, workspace,
                                      stream=stream)
        for u in self.adamw_units:
            fsdp_zero1_adamw_broadcast(self.layout, u, u + 1, grads, self.master, self.exp_avg, self.exp_avg_sq, self.params, adamw, t,
                                       stream)
        self.t = t
