"""fsdp_sharded_state_gb300 -- the FSDP / ZeRO-3 sharded-state step on one GB300.

Thin ctypes binding of ``libfsdpstate.so`` (C ABI in ``include/fsdp_state.h``).
The functions here carry the C names and only marshal arguments: torch tensors
(or raw device pointers) in, status codes checked, ``FsdpError`` out.  Every step
of the path runs in the library's CUDA kernels; there is no CPU fallback -- if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libfsdpstate.so")

FSDP_FLAT, FSDP_DIM0, FSDP_ZERO1 = 0, 1, 2
FSDP_F32, FSDP_BF16 = 0, 1
MODES = {"flat": FSDP_FLAT, "dim0": FSDP_DIM0, "zero1": FSDP_ZERO1}

FSDP_RS_AUTO, FSDP_RS_DIRECT, FSDP_RS_STAGED = 0, 1, 2
RS_KERNELS = {"auto": FSDP_RS_AUTO, "direct": FSDP_RS_DIRECT, "staged": FSDP_RS_STAGED}

FSDP_OK = 0
STATUS = {0: "FSDP_OK", -1: "FSDP_EINVAL", -2: "FSDP_EDTYPE", -3: "FSDP_ESHAPE", -4: "FSDP_EALIGN",
          -5: "FSDP_EOVERFLOW", -6: "FSDP_ECUDA", -7: "FSDP_ETIMEOUT", -8: "FSDP_ENOMEM"}

# Every symbol include/fsdp_state.h declares.
EXPORTS = ("fsdp_layout_create", "fsdp_layout_destroy", "fsdp_layout_query", "fsdp_layout_unit",
           "fsdp_layout_tensor", "fsdp_layout_segment", "fsdp_state_bytes", "fsdp_layout_prepare",
           "fsdp_unshard", "fsdp_reduce_scatter_adamw", "fsdp_reshard", "fsdp_check_status",
           "fsdp_error_string", "fsdp_last_cuda_error", "fsdp_reduce_scatter_adamw_noalloc",
           "fsdp_layout_owner", "fsdp_clip_workspace_bytes", "fsdp_reduce_scatter_clip_adamw",
           "fsdp_accumulate_grads", "fsdp_hsdp_reduce_scatter_adamw", "fsdp_zero1_adamw_broadcast",
           "fsdp_set_rs_kernel", "fsdp_rs_kernel_for", "fsdp_wait_selftest", "fsdp_adamw_step_consts_make",
           "fsdp_reduce_scatter_adamw_consts", "fsdp_adamw_step_consts_upload", "fsdp_collective_payload",
           "fsdp_accumulate_reduce_scatter_adamw", "fsdp_linear_workspace_bytes", "fsdp_linear_forward",
           "fsdp_linear_dgrad", "fsdp_linear_wgrad", "fsdp_dropout", "fsdp_layernorm_forward",
           "fsdp_layernorm_workspace_bytes", "fsdp_layernorm_backward", "fsdp_newton_schulz",
           "fsdp_newton_schulz_workspace_bytes", "fsdp_zero1_muon_broadcast", "fsdp_zero1_muon_workspace_bytes")


class FsdpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        if status == -6 and _lib is not None:
            msg += f" ({_lib.fsdp_last_cuda_error().decode()})"
        super().__init__(msg)


class LayoutInfo(C.Structure):
    _fields_ = [("n_tensors", C.c_int32), ("n_units", C.c_int32), ("n_ranks", C.c_int32), ("mode", C.c_int32),
                ("numel", C.c_int64), ("shard_numel", C.c_int64), ("shard_stride", C.c_int64),
                ("full_numel", C.c_int64), ("pad_numel", C.c_int64), ("n_segments", C.c_int64)]


FSDP_NO_SHARD, FSDP_ZERO1_OPT, FSDP_SHARD_GRAD_OP, FSDP_FULL_SHARD, FSDP_HYBRID_SHARD = 0, 1, 2, 3, 4
STRATEGIES = {"no_shard": FSDP_NO_SHARD, "zero1": FSDP_ZERO1_OPT, "shard_grad_op": FSDP_SHARD_GRAD_OP,
              "full_shard": FSDP_FULL_SHARD, "hybrid_shard": FSDP_HYBRID_SHARD}


class CollectivePayload(C.Structure):
    _fields_ = [("allreduce_input", C.c_int64), ("forward_allgather", C.c_int64),
                ("backward_allgather", C.c_int64), ("reducescatter_input", C.c_int64), ("broadcast", C.c_int64),
                ("bus_elements", C.c_double)]


class AdamWHparams(C.Structure):
    _fields_ = [("lr", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float),
                ("weight_decay", C.c_float)]


class AdamWStepConsts(C.Structure):
    """The 48-byte block of per-step AdamW constants (fsdp_adamw_step_consts)."""
    _fields_ = [("decay", C.c_float), ("om1", C.c_float), ("om2", C.c_float), ("step_size", C.c_float),
                ("bc2s", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float),
                ("n_avg", C.c_float), ("reserved", C.c_float * 3)]


MUON_SCALES = {"none": 0, "shape": 1, "rms": 2}


class MuonHparams(C.Structure):
    """Hyper-parameters of the Muon step (fsdp_muon_hparams).  scale: "none" (1), "shape"
    (sqrt(max(1, rows / cols))) or "rms" (0.2 sqrt(max(rows, cols)))."""
    _fields_ = [("lr", C.c_float), ("momentum", C.c_float), ("weight_decay", C.c_float), ("eps", C.c_float),
                ("nesterov", C.c_int32), ("steps", C.c_int32), ("scale", C.c_int32), ("reserved", C.c_int32)]

    def __init__(self, lr: float = 0.02, momentum: float = 0.95, weight_decay: float = 0.0, eps: float = 1e-7,
                 nesterov: bool = True, steps: int = 5, scale="rms"):
        code = MUON_SCALES.get(scale) if isinstance(scale, str) else int(scale)
        if code is None:
            raise ValueError(f"unknown scale {scale!r}: {sorted(MUON_SCALES)}")
        super().__init__(lr, momentum, weight_decay, eps, int(bool(nesterov)), steps, code, 0)


FSDP_ACT_NONE, FSDP_ACT_RELU, FSDP_ACT_GELU, FSDP_ACT_SILU = 0, 1, 2, 3
ACTIVATIONS = {"none": FSDP_ACT_NONE, "relu": FSDP_ACT_RELU, "gelu": FSDP_ACT_GELU, "silu": FSDP_ACT_SILU}


class DropoutSpec(C.Structure):
    """A dropout with a mask drawn from (seed, layer, row, column) (fsdp_dropout_spec);
    row0 is the index of the first row of a call's matrix in the whole batch."""
    _fields_ = [("p", C.c_double), ("seed", C.c_uint64), ("row0", C.c_int64), ("layer", C.c_uint32),
                ("reserved", C.c_uint32)]

    def __init__(self, p: float, seed: int, layer: int = 0, row0: int = 0):
        super().__init__(float(p), seed, row0, layer, 0)


_lib: Optional[C.CDLL] = None


def lib() -> C.CDLL:
    """The loaded libfsdpstate; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfsdpstate is not built ({LIB_PATH} missing): run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` first")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
        L.fsdp_layout_create.argtypes = [i32, vp, vp, vp, vp, i32, i32, C.POINTER(vp)]
        L.fsdp_layout_destroy.argtypes = [vp]
        L.fsdp_layout_destroy.restype = None
        L.fsdp_layout_query.argtypes = [vp, C.POINTER(LayoutInfo)]
        L.fsdp_layout_unit.argtypes = [vp, i32] + [C.POINTER(i64)] * 5
        L.fsdp_layout_tensor.argtypes = [vp, i32, C.POINTER(i32)] + [C.POINTER(i64)] * 4
        L.fsdp_layout_segment.argtypes = [vp, i32, i32] + [C.POINTER(i64)] * 4
        L.fsdp_state_bytes.argtypes = [vp, i32, i32, i32, i64, i64, i64, i64, C.POINTER(i64)]
        L.fsdp_collective_payload.argtypes = [vp, i32, i32, C.POINTER(CollectivePayload)]
        L.fsdp_layout_prepare.argtypes = [vp]
        L.fsdp_unshard.argtypes = [vp, i32, i32, vp, vp, i32, vp]
        L.fsdp_reduce_scatter_adamw.argtypes = [vp, i32, i32, C.POINTER(vp), i32, vp, vp, vp, vp, vp,
                                                C.POINTER(AdamWHparams), i64, vp]
        L.fsdp_reshard.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp]
        L.fsdp_reduce_scatter_adamw_noalloc.argtypes = L.fsdp_reduce_scatter_adamw.argtypes
        L.fsdp_layout_owner.argtypes = [vp, i32, C.POINTER(i32)]
        L.fsdp_clip_workspace_bytes.argtypes = []
        L.fsdp_clip_workspace_bytes.restype = C.c_size_t
        L.fsdp_reduce_scatter_clip_adamw.argtypes = [vp, i32, i32, C.POINTER(vp), i32, vp, vp, vp, vp, vp, C.c_float,
                                                     vp, vp, C.POINTER(AdamWHparams), i64, vp]
        L.fsdp_accumulate_grads.argtypes = [vp, i32, i32, C.POINTER(vp), C.POINTER(vp), i32, i32, vp]
        L.fsdp_accumulate_reduce_scatter_adamw.argtypes = [vp, i32, i32, C.POINTER(vp), C.POINTER(vp), i32, vp, vp,
                                                           vp, vp, vp, C.POINTER(AdamWHparams), i64, vp]
        L.fsdp_hsdp_reduce_scatter_adamw.argtypes = [vp, i32, i32, i32, C.POINTER(vp), i32, vp, vp, vp, vp,
                                                     C.POINTER(AdamWHparams), i64, vp]
        L.fsdp_zero1_adamw_broadcast.argtypes = [vp, i32, i32, C.POINTER(vp), i32, vp, vp, vp, C.POINTER(vp), i32,
                                                 C.POINTER(AdamWHparams), i64, vp]
        sz, drop = C.c_size_t, C.POINTER(DropoutSpec)
        L.fsdp_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
        L.fsdp_linear_workspace_bytes.restype = sz
        L.fsdp_linear_forward.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i32, drop, vp, i64, vp, i64, vp,
                                          i64, vp, sz, vp]
        L.fsdp_linear_dgrad.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, i32, vp, i64, drop, vp, i64, vp, i64,
                                        vp, sz, vp]
        L.fsdp_linear_wgrad.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, vp, i64, vp, i32, i32, vp, sz, vp]
        L.fsdp_dropout.argtypes = [i64, i64, i32, vp, i64, drop, vp, i64, vp, i64, vp]
        L.fsdp_layernorm_forward.argtypes = [i64, i64, i32, vp, i64, vp, vp, C.c_float, vp, i64, vp, vp, vp]
        L.fsdp_layernorm_workspace_bytes.argtypes = [i64, i64]
        L.fsdp_layernorm_workspace_bytes.restype = sz
        L.fsdp_layernorm_backward.argtypes = [i64, i64, i32, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, i32, i32, vp,
                                              sz, vp]
        L.fsdp_newton_schulz.argtypes = [i32, i64, i64, vp, vp, i32, vp, vp, i32, i32, vp, C.c_float, vp, sz, vp]
        L.fsdp_newton_schulz_workspace_bytes.argtypes = [i32, i64, i64]
        L.fsdp_newton_schulz_workspace_bytes.restype = sz
        L.fsdp_zero1_muon_broadcast.argtypes = [vp, i32, vp, C.POINTER(vp), i32, vp, vp, C.POINTER(vp), i32, C.POINTER(MuonHparams), vp,
                                                vp, sz, vp]
        L.fsdp_zero1_muon_workspace_bytes.argtypes = [vp, i32, vp]
        L.fsdp_zero1_muon_workspace_bytes.restype = sz
        L.fsdp_check_status.argtypes = [vp]
        L.fsdp_set_rs_kernel.argtypes = [i32]
        L.fsdp_rs_kernel_for.argtypes = [vp, i32]
        L.fsdp_wait_selftest.argtypes = [i64, vp]
        L.fsdp_adamw_step_consts_make.argtypes = [vp, C.POINTER(AdamWHparams), i64, C.POINTER(AdamWStepConsts)]
        L.fsdp_reduce_scatter_adamw_consts.argtypes = [vp, i32, i32, C.POINTER(vp), i32, vp, vp, vp, vp, vp, vp, vp]
        L.fsdp_adamw_step_consts_upload.argtypes = [vp, vp, vp]
        L.fsdp_error_string.argtypes = [C.c_int]
        L.fsdp_error_string.restype = C.c_char_p
        L.fsdp_last_cuda_error.argtypes = []
        L.fsdp_last_cuda_error.restype = C.c_char_p
        _lib = L
    return _lib


def _check(rc: int, where: str) -> None:
    if rc != FSDP_OK:
        raise FsdpError(rc, where)


def _ptr(x) -> Optional[int]:
    """Device address of a tensor (or an int address); None stays NULL."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("buffers must be contiguous")
    return x.data_ptr()


# The raw handle alone: a Stream object costs 3 us.  torch keeps this call to itself, so it may go.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None) -> Optional[int]:
    """A stream's handle; None: the current one (of the current device, where its index is known)."""
    if stream is None:
        if _raw_stream is not None and (device is not None or torch.cuda.is_initialized()):
            return _raw_stream(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_DTYPE_CODES = {torch.float32: FSDP_F32, torch.bfloat16: FSDP_BF16}


def _dtype_code(t) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")
    return code


class Layout:
    """An fsdp_layout: shapes + unit ids + N + mode -> offsets, padding, segments."""

    def __init__(self, shapes: Sequence[Sequence[int]], unit_ids: Optional[Sequence[int]] = None,
                 n_ranks: int = 1, mode: int = FSDP_FLAT, dtypes: Optional[Sequence[int]] = None):
        shapes = [tuple(int(d) for d in s) for s in shapes]
        T = len(shapes)
        if unit_ids is None:
            unit_ids = [0] * T
        ndim = (C.c_int32 * max(T, 1))(*[len(s) for s in shapes])
        flat = [d for s in shapes for d in s] or [0]
        dims = (C.c_int64 * len(flat))(*flat)
        units = (C.c_int32 * max(T, 1))(*unit_ids)
        dt = None if dtypes is None else (C.c_int32 * max(T, 1))(*dtypes)
        h = C.c_void_p()
        self._h = None
        _check(lib().fsdp_layout_create(T, ndim, dims, units, dt, n_ranks, mode, C.byref(h)),
               "fsdp_layout_create")
        self._h = h
        self.shapes, self.unit_ids, self.n_ranks, self.mode = shapes, list(unit_ids), n_ranks, mode
        info = LayoutInfo()
        _check(lib().fsdp_layout_query(self._h, C.byref(info)), "fsdp_layout_query")
        self.info = {k: getattr(info, k) for k, _ in LayoutInfo._fields_}

    # -- queries --------------------------------------------------------------
    @property
    def handle(self):
        return self._h

    @property
    def N(self) -> int:
        return self.info["n_ranks"]

    @property
    def stride(self) -> int:
        return self.info["shard_stride"]

    @property
    def n_units(self) -> int:
        return self.info["n_units"]

    def unit(self, u: int) -> dict:
        v = [C.c_int64() for _ in range(5)]
        _check(lib().fsdp_layout_unit(self._h, u, *[C.byref(x) for x in v]), "fsdp_layout_unit")
        return dict(zip(("shard_off", "shard_numel", "full_off", "full_numel", "numel"), (x.value for x in v)))

    def tensor(self, t: int) -> dict:
        u = C.c_int32()
        v = [C.c_int64() for _ in range(4)]
        _check(lib().fsdp_layout_tensor(self._h, t, C.byref(u), *[C.byref(x) for x in v]), "fsdp_layout_tensor")
        d = dict(zip(("numel", "full_off", "shard_off", "rows_per_rank"), (x.value for x in v)))
        d["unit"] = u.value
        return d

    def segment(self, t: int, r: int) -> dict:
        v = [C.c_int64() for _ in range(4)]
        _check(lib().fsdp_layout_segment(self._h, t, r, *[C.byref(x) for x in v]), "fsdp_layout_segment")
        return dict(zip(("shard_off", "full_off", "len", "pad"), (x.value for x in v)))

    def owner(self, t: int) -> int:
        r = C.c_int32()
        _check(lib().fsdp_layout_owner(self._h, t, C.byref(r)), "fsdp_layout_owner")
        return r.value

    def state_bytes(self, stage: int, rank: int, physical: bool, param_bytes: int, grad_bytes: int,
                    optim_bytes: int, step_bytes: int = 0):
        out = (C.c_int64 * 3)()
        _check(lib().fsdp_state_bytes(self._h, stage, rank, int(physical), param_bytes, grad_bytes, optim_bytes,
                                      step_bytes, out), "fsdp_state_bytes")
        return tuple(out)

    def collective_payload(self, strategy, n_groups: int = 1) -> dict:
        """Per-rank collective payload of one step (fsdp_collective_payload): logical
        input elements of each collective and the ring bus elements a rank sends."""
        code = STRATEGIES[strategy] if isinstance(strategy, str) else int(strategy)
        out = CollectivePayload()
        _check(lib().fsdp_collective_payload(self._h, code, n_groups, C.byref(out)), "fsdp_collective_payload")
        return {f: getattr(out, f) for f, _ in CollectivePayload._fields_}

    def prepare(self) -> None:
        _check(lib().fsdp_layout_prepare(self._h), "fsdp_layout_prepare")

    def close(self) -> None:
        if self._h is not None and _lib is not None:
            _lib.fsdp_layout_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# -- the C names ----------------------------------------------------------------
def fsdp_layout_create(shapes, unit_ids=None, n_ranks=1, mode=FSDP_FLAT, dtypes=None) -> Layout:
    return Layout(shapes, unit_ids, n_ranks, mode, dtypes)


def fsdp_unshard(layout: Layout, unit_begin: int, unit_end: int, param_shards, full, stream=None,
                 elem_dtype: Optional[int] = None) -> None:
    if elem_dtype is None:
        elem_dtype = _dtype_code(param_shards)
    _check(lib().fsdp_unshard(layout.handle, unit_begin, unit_end, _ptr(param_shards), _ptr(full), elem_dtype,
                              _stream(stream)), "fsdp_unshard")


def fsdp_reduce_scatter_adamw(layout: Layout, unit_begin: int, unit_end: int, grad_replicas, master, exp_avg,
                              exp_avg_sq, param_shards=None, grad_shard_out=None,
                              hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1, stream=None,
                              grad_dtype: Optional[int] = None) -> None:
    if len(grad_replicas) != layout.N:
        raise ValueError(f"need {layout.N} gradient replicas, got {len(grad_replicas)}")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    arr = (C.c_void_p * layout.N)(*[_ptr(g) for g in grad_replicas])
    h = hp if isinstance(hp, AdamWHparams) else AdamWHparams(*hp)
    _check(lib().fsdp_reduce_scatter_adamw(layout.handle, unit_begin, unit_end, arr, grad_dtype, _ptr(master),
                                           _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(param_shards),
                                           _ptr(grad_shard_out), C.byref(h), step, _stream(stream)),
           "fsdp_reduce_scatter_adamw")


def fsdp_reduce_scatter_adamw_noalloc(layout: Layout, unit_begin: int, unit_end: int, grad_replicas, master,
                                      exp_avg, exp_avg_sq, param_shards=None, grad_shard_out=None,
                                      hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1, stream=None,
                                      grad_dtype: Optional[int] = None) -> None:
    """fsdp_reduce_scatter_adamw without any device allocation (fixed in-library scratch)."""
    if len(grad_replicas) != layout.N:
        raise ValueError(f"need {layout.N} gradient replicas, got {len(grad_replicas)}")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    arr = (C.c_void_p * layout.N)(*[_ptr(g) for g in grad_replicas])
    h = hp if isinstance(hp, AdamWHparams) else AdamWHparams(*hp)
    _check(lib().fsdp_reduce_scatter_adamw_noalloc(layout.handle, unit_begin, unit_end, arr, grad_dtype,
                                                   _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq),
                                                   _ptr(param_shards), _ptr(grad_shard_out), C.byref(h), step,
                                                   _stream(stream)), "fsdp_reduce_scatter_adamw_noalloc")


def fsdp_adamw_step_consts_make(layout: Layout, hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1) -> AdamWStepConsts:
    """The step's AdamW constants as the fused step forms them (host only)."""
    out = AdamWStepConsts()
    h = hp if isinstance(hp, AdamWHparams) else AdamWHparams(*hp)
    _check(lib().fsdp_adamw_step_consts_make(layout.handle, C.byref(h), step, C.byref(out)),
           "fsdp_adamw_step_consts_make")
    return out


def fsdp_adamw_step_consts_upload(dev_dst, host_src, stream=None) -> None:
    """Copies a 48-byte block of step constants from (pinned) host memory to the device
    block on the stream; inside a CUDA graph capture it reads host_src at every replay."""
    _check(lib().fsdp_adamw_step_consts_upload(_ptr(dev_dst), _ptr(host_src), _stream(stream)),
           "fsdp_adamw_step_consts_upload")


def fsdp_reduce_scatter_adamw_consts(layout: Layout, unit_begin: int, unit_end: int, grad_replicas, master,
                                     exp_avg, exp_avg_sq, param_shards=None, grad_shard_out=None, consts=None,
                                     stream=None, grad_dtype: Optional[int] = None) -> None:
    """fsdp_reduce_scatter_adamw with the step constants read on the device from `consts`
    (a 48-byte device buffer, e.g. a float32 tensor of 12 elements)."""
    if len(grad_replicas) != layout.N:
        raise ValueError(f"need {layout.N} gradient replicas, got {len(grad_replicas)}")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    arr = (C.c_void_p * layout.N)(*[_ptr(g) for g in grad_replicas])
    _check(lib().fsdp_reduce_scatter_adamw_consts(layout.handle, unit_begin, unit_end, arr, grad_dtype,
                                                  _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq),
                                                  _ptr(param_shards), _ptr(grad_shard_out), _ptr(consts),
                                                  _stream(stream)), "fsdp_reduce_scatter_adamw_consts")


def _ptr_array(xs):
    return (C.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def _hp(hp):
    return hp if isinstance(hp, AdamWHparams) else AdamWHparams(*hp)


def fsdp_clip_workspace_bytes() -> int:
    return int(lib().fsdp_clip_workspace_bytes())


def fsdp_reduce_scatter_clip_adamw(layout: Layout, unit_begin: int, unit_end: int, grad_replicas, master, exp_avg,
                                   exp_avg_sq, param_shards, grad_shard, max_norm: float, workspace,
                                   norm_out=None, hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1,
                                   stream=None, grad_dtype: Optional[int] = None) -> None:
    if len(grad_replicas) != layout.N:
        raise ValueError(f"need {layout.N} gradient replicas, got {len(grad_replicas)}")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    _check(lib().fsdp_reduce_scatter_clip_adamw(layout.handle, unit_begin, unit_end, _ptr_array(grad_replicas),
                                                grad_dtype, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq),
                                                _ptr(param_shards), _ptr(grad_shard), float(max_norm),
                                                _ptr(workspace), _ptr(norm_out), C.byref(_hp(hp)), step,
                                                _stream(stream)), "fsdp_reduce_scatter_clip_adamw")


def fsdp_accumulate_grads(layout: Layout, unit_begin: int, unit_end: int, acc, micro, first: bool,
                          stream=None, micro_dtype: Optional[int] = None) -> None:
    if len(acc) != layout.N or len(micro) != layout.N:
        raise ValueError(f"need {layout.N} accumulators and micro-gradients")
    if micro_dtype is None:
        micro_dtype = _dtype_code(micro[0])
    _check(lib().fsdp_accumulate_grads(layout.handle, unit_begin, unit_end, _ptr_array(acc), _ptr_array(micro),
                                       micro_dtype, int(bool(first)), _stream(stream)), "fsdp_accumulate_grads")


def fsdp_accumulate_reduce_scatter_adamw(layout: Layout, unit_begin: int, unit_end: int, acc, micro, master,
                                         exp_avg, exp_avg_sq, param_shards=None, grad_shard_out=None,
                                         hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1, stream=None,
                                         micro_dtype: Optional[int] = None) -> None:
    """The last micro-batch of a no_sync accumulation fused with the step: acc (N fp32
    accumulators, read only) plus micro (N micro-batch gradients), reduce-scattered, AdamW, cast."""
    if len(acc) != layout.N or len(micro) != layout.N:
        raise ValueError(f"need {layout.N} accumulators and micro-gradients")
    if micro_dtype is None:
        micro_dtype = _dtype_code(micro[0])
    h = hp if isinstance(hp, AdamWHparams) else AdamWHparams(*hp)
    _check(lib().fsdp_accumulate_reduce_scatter_adamw(layout.handle, unit_begin, unit_end, _ptr_array(acc),
                                                      _ptr_array(micro), micro_dtype, _ptr(master), _ptr(exp_avg),
                                                      _ptr(exp_avg_sq), _ptr(param_shards), _ptr(grad_shard_out),
                                                      C.byref(h), step, _stream(stream)),
           "fsdp_accumulate_reduce_scatter_adamw")


def fsdp_hsdp_reduce_scatter_adamw(layout: Layout, unit_begin: int, unit_end: int, n_groups: int, grad_replicas,
                                   master, exp_avg, exp_avg_sq, param_shards=None,
                                   hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1, stream=None,
                                   grad_dtype: Optional[int] = None) -> None:
    if len(grad_replicas) != layout.N * n_groups:
        raise ValueError(f"need {layout.N * n_groups} gradient replicas, got {len(grad_replicas)}")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    _check(lib().fsdp_hsdp_reduce_scatter_adamw(layout.handle, unit_begin, unit_end, n_groups,
                                                _ptr_array(grad_replicas), grad_dtype, _ptr(master), _ptr(exp_avg),
                                                _ptr(exp_avg_sq), _ptr(param_shards), C.byref(_hp(hp)), step,
                                                _stream(stream)), "fsdp_hsdp_reduce_scatter_adamw")


def fsdp_zero1_adamw_broadcast(layout: Layout, unit_begin: int, unit_end: int, grad_replicas, master, exp_avg,
                               exp_avg_sq, param_replicas, hp=(1e-3, 0.9, 0.999, 1e-8, 0.01), step: int = 1,
                               stream=None, grad_dtype: Optional[int] = None,
                               param_dtype: Optional[int] = None) -> None:
    if len(grad_replicas) != layout.N or len(param_replicas) != layout.N:
        raise ValueError(f"need {layout.N} gradient and parameter replicas")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    if param_dtype is None:
        param_dtype = _dtype_code(param_replicas[0])
    _check(lib().fsdp_zero1_adamw_broadcast(layout.handle, unit_begin, unit_end, _ptr_array(grad_replicas),
                                            grad_dtype, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq),
                                            _ptr_array(param_replicas), param_dtype, C.byref(_hp(hp)), step,
                                            _stream(stream)), "fsdp_zero1_adamw_broadcast")


# -- layers between the all-gather and the reduce-scatter -------------------------
# All tensors of a call, its workspace too, lie on the current device.
def _refuse_device(x, name: str, device) -> None:
    if not x.is_cuda:
        raise ValueError(f"{name} is not a CUDA tensor")
    at = x.get_device()
    if device is None:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{torch.cuda.current_device()}")
    raise ValueError(f"{name} is on cuda:{at}, the first operand on cuda:{device}")


def _device(x):
    """The device of a call's first tensor, where all others have to be: the current one, else None."""
    at = x.get_device()
    return at if at >= 0 and at == torch.cuda.current_device() else None


def _operand(x, name: str, dtype, device):
    """(rows, cols, address, row stride) of a matrix on the device whose rows are contiguous."""
    if x.dtype is not dtype:
        raise TypeError(f"{name} is {x.dtype}, expected {dtype}")
    if x.dim() != 2:
        raise ValueError(f"{name} is {tuple(x.shape)}, expected a matrix")
    if x.get_device() != device:
        _refuse_device(x, name, device)
    rows, cols = x.shape
    ld, one = x.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: a row's elements must be contiguous")
    if rows <= 1 and ld < cols:
        ld = cols                                # torch leaves a single row's stride arbitrary
    return rows, cols, x.data_ptr(), ld


def _matrix(x, name: str, rows: int, cols: int, dtype, device):
    """(address, row stride) of such a matrix of the given shape."""
    r, c, p, ld = _operand(x, name, dtype, device)
    if r != rows or c != cols:
        raise ValueError(f"{name} is {tuple(x.shape)}, expected {(rows, cols)}")
    return p, ld


_NO_MATRIX = (None, 0)


def _vector(x, name: str, n: int, dtype, device):
    if x.dtype is not dtype:
        raise TypeError(f"{name} is {x.dtype}, expected {dtype}")
    if x.shape != (n,):
        raise ValueError(f"{name} is {tuple(x.shape)}, expected {(n,)}")
    if x.get_device() != device:
        _refuse_device(x, name, device)
    if n > 1 and x.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


def _act(act) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        if isinstance(act, str):
            raise ValueError(f"unknown activation {act!r}: {sorted(ACTIVATIONS)}")
        code = int(act)
    return code


def _workspace(ws, device):
    if ws.get_device() != device:
        _refuse_device(ws, "workspace", device)
    return (_ptr(ws), ws.numel() * ws.element_size())


def _drop(spec):
    return None if spec is None else C.byref(spec)


def fsdp_linear_workspace_bytes(rows: int, cols_in: int, cols_out: int, dtype, aligned: Optional[bool] = None) -> int:
    """Scratch bytes of the three linear calls at these sizes.  aligned: every x, w and dz
    has a base address and row stride that are multiples of 16 bytes (default: widths of
    whole 16-byte rows, as contiguous tensors of their own have)."""
    code = dtype if isinstance(dtype, int) else {torch.float32: FSDP_F32, torch.bfloat16: FSDP_BF16}[dtype]
    if aligned is None:
        e = 4 if code == FSDP_F32 else 2
        aligned = cols_in * e % 16 == 0 and cols_out * e % 16 == 0
    return int(lib().fsdp_linear_workspace_bytes(rows, cols_in, cols_out, code, int(aligned)))


def fsdp_linear_forward(x, w, y, bias=None, act="none", preact=None, dropout: Optional[DropoutSpec] = None,
                        residual=None, workspace=None, stream=None) -> None:
    """y = residual + drop(act(x w^T + bias)); z = x w^T + bias into preact where given.
    x [rows, in], w [out, in], y / preact / residual [rows, out], bias [out], one dtype."""
    code, dt, dev = _dtype_code(x), x.dtype, _device(x)
    rows, cin, px, ldx = _operand(x, "x", dt, dev)
    cout, wcols, pw, ldw = _operand(w, "w", dt, dev)
    if wcols != cin:
        raise ValueError(f"w is {tuple(w.shape)}, expected {(cout, cin)}")
    py, ldy = _matrix(y, "y", rows, cout, dt, dev)
    pr, ldr = _NO_MATRIX if residual is None else _matrix(residual, "residual", rows, cout, dt, dev)
    pz, ldz = _NO_MATRIX if preact is None else _matrix(preact, "preact", rows, cout, dt, dev)
    pb = None if bias is None else _vector(bias, "bias", cout, dt, dev)
    pws, nws = _NO_MATRIX if workspace is None else _workspace(workspace, dev)
    rc = lib().fsdp_linear_forward(rows, cin, cout, code, px, ldx, pw, ldw, pb, _act(act), _drop(dropout), pr, ldr, py, ldy,
                                   pz, ldz, pws, nws, _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_linear_forward")


def fsdp_linear_dgrad(dz, w, dx, act="none", preact=None, dropout: Optional[DropoutSpec] = None, residual=None,
                      workspace=None, stream=None) -> None:
    """dx = residual + act'(preact) * drop(dz w): dz [rows, out], w [out, in], dx / preact /
    residual [rows, in]; act, preact and dropout are those of the layer before."""
    code, dt, dev = _dtype_code(dz), dz.dtype, _device(dz)
    rows, cout, pg, ldg = _operand(dz, "dz", dt, dev)
    wrows, cin, pw, ldw = _operand(w, "w", dt, dev)
    if wrows != cout:
        raise ValueError(f"w is {tuple(w.shape)}, expected {(cout, cin)}")
    px, ldx = _matrix(dx, "dx", rows, cin, dt, dev)
    pz, ldz = _NO_MATRIX if preact is None else _matrix(preact, "preact", rows, cin, dt, dev)
    pr, ldr = _NO_MATRIX if residual is None else _matrix(residual, "residual", rows, cin, dt, dev)
    pws, nws = _NO_MATRIX if workspace is None else _workspace(workspace, dev)
    rc = lib().fsdp_linear_dgrad(rows, cin, cout, code, pg, ldg, pw, ldw, _act(act), pz, ldz, _drop(dropout), pr, ldr, px,
                                 ldx, pws, nws, _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_linear_dgrad")


def fsdp_linear_wgrad(dz, x, dw, db=None, accumulate: bool = False, workspace=None, stream=None) -> None:
    """dw (+)= dz^T x and db (+)= the column sums of dz: dz [rows, out], x [rows, in] of one
    dtype, dw [out, in] and db [out] of one dtype (a gradient replica's, or fp32)."""
    code, dt, dev = _dtype_code(dz), dz.dtype, _device(dz)
    rows, cout, pg, ldg = _operand(dz, "dz", dt, dev)
    xrows, cin, px, ldx = _operand(x, "x", dt, dev)
    if xrows != rows:
        raise ValueError(f"x is {tuple(x.shape)}, expected {(rows, cin)}")
    pw, ldw = _matrix(dw, "dw", cout, cin, dw.dtype, dev)
    pb = None if db is None else _vector(db, "db", cout, dw.dtype, dev)
    pws, nws = _NO_MATRIX if workspace is None else _workspace(workspace, dev)
    rc = lib().fsdp_linear_wgrad(rows, cin, cout, code, pg, ldg, px, ldx, pw, ldw, pb, _dtype_code(dw), 1 if accumulate else 0,
                                 pws, nws, _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_linear_wgrad")


def fsdp_dropout(x, y, dropout: Optional[DropoutSpec], residual=None, stream=None) -> None:
    """y = residual + drop(x), [rows, cols] each; the same call on the gradient is its backward."""
    code, dt, dev = _dtype_code(x), x.dtype, _device(x)
    rows, cols, px, ldx = _operand(x, "x", dt, dev)
    py, ldy = _matrix(y, "y", rows, cols, dt, dev)
    pr, ldr = _NO_MATRIX if residual is None else _matrix(residual, "residual", rows, cols, dt, dev)
    rc = lib().fsdp_dropout(rows, cols, code, px, ldx, _drop(dropout), pr, ldr, py, ldy, _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_dropout")


def fsdp_layernorm_forward(x, y, weight=None, bias=None, mean=None, rstd=None, eps: float = 1e-5, stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias per row: x, y [rows, cols], weight and bias [cols], one
    dtype; the rows' mean and rstd [rows], float32, are written where given."""
    code, dt, dev = _dtype_code(x), x.dtype, _device(x)
    rows, cols, px, ldx = _operand(x, "x", dt, dev)
    py, ldy = _matrix(y, "y", rows, cols, dt, dev)
    pw = None if weight is None else _vector(weight, "weight", cols, dt, dev)
    pb = None if bias is None else _vector(bias, "bias", cols, dt, dev)
    pm = None if mean is None else _vector(mean, "mean", rows, torch.float32, dev)
    pr = None if rstd is None else _vector(rstd, "rstd", rows, torch.float32, dev)
    rc = lib().fsdp_layernorm_forward(rows, cols, code, px, ldx, pw, pb, eps, py, ldy, pm, pr, _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_layernorm_forward")


def fsdp_layernorm_workspace_bytes(rows: int, cols: int) -> int:
    """Scratch bytes of fsdp_layernorm_backward with dw or db."""
    return int(lib().fsdp_layernorm_workspace_bytes(rows, cols))


def fsdp_layernorm_backward(dy, x, mean, rstd, dx, weight=None, dw=None, db=None, residual=None, accumulate: bool = False,
                            workspace=None, stream=None) -> None:
    """dx = residual + the gradient of x from that of y; dw (+)= the sums over rows of dy (x - mean)
    rstd, db (+)= those of dy: dy, x, dx, residual [rows, cols] and weight [cols] of one dtype, mean
    and rstd [rows] float32 as forward wrote them, dw and db [cols] of one dtype (a gradient
    replica's, or fp32)."""
    code, dt, dev = _dtype_code(dy), dy.dtype, _device(dy)
    rows, cols, pg, ldg = _operand(dy, "dy", dt, dev)
    px, ldx = _matrix(x, "x", rows, cols, dt, dev)
    pm, pr = _vector(mean, "mean", rows, torch.float32, dev), _vector(rstd, "rstd", rows, torch.float32, dev)
    po, ldo = _matrix(dx, "dx", rows, cols, dt, dev)
    pw = None if weight is None else _vector(weight, "weight", cols, dt, dev)
    ps, lds = _NO_MATRIX if residual is None else _matrix(residual, "residual", rows, cols, dt, dev)
    first = dw if dw is not None else db
    gcode = code if first is None else _dtype_code(first)
    pdw = None if dw is None else _vector(dw, "dw", cols, first.dtype, dev)
    pdb = None if db is None else _vector(db, "db", cols, first.dtype, dev)
    pws, nws = _NO_MATRIX if workspace is None else _workspace(workspace, dev)
    rc = lib().fsdp_layernorm_backward(rows, cols, code, pg, ldg, px, ldx, pm, pr, pw, ps, lds, po, ldo, pdw, pdb, gcode,
                                       1 if accumulate else 0, pws, nws, _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_layernorm_backward")


def _coeffs(coeffs, steps: int):
    """A schedule of (a, b, c) per step as a C array; None: the default."""
    if coeffs is None:
        return None
    rows = [tuple(map(float, r)) for r in coeffs]
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError(f"coeffs: need (a, b, c) for each of {steps} steps")
    return (C.c_float * (3 * steps))(*[v for r in rows for v in r])


def fsdp_newton_schulz_workspace_bytes(count: int, rows: int, cols: int) -> int:
    """Scratch bytes of fsdp_newton_schulz for `count` matrices of rows x cols."""
    return int(lib().fsdp_newton_schulz_workspace_bytes(count, rows, cols))


def fsdp_newton_schulz(src, dst, steps: int = 5, coeffs=None, eps: float = 1e-7, workspace=None, stream=None) -> None:
    """dst = src / |src| after `steps` Newton-Schulz steps X <- a X + (b A + c A A) X, A = X X^T (or of the
    transpose, where that has fewer rows): a matrix, or a list of matrices of one shape; src of one
    dtype, dst of one dtype.  coeffs: (a, b, c) per step.  workspace:
    fsdp_newton_schulz_workspace_bytes."""
    if isinstance(src, torch.Tensor):
        src, dst = [src], [dst]
    n = len(src)
    if len(dst) != n:
        raise ValueError(f"{n} sources, {len(dst)} destinations")
    if n == 0:
        return
    code, dev = _dtype_code(src[0]), _device(src[0])
    rows, cols, _, _ = _operand(src[0], "src", src[0].dtype, dev)
    out = _dtype_code(dst[0])
    a = [_matrix(x, "src", rows, cols, src[0].dtype, dev) for x in src]
    b = [_matrix(x, "dst", rows, cols, dst[0].dtype, dev) for x in dst]
    pa, la = (C.c_void_p * n)(*[p for p, _ in a]), (C.c_int64 * n)(*[ld for _, ld in a])
    pb, lb = (C.c_void_p * n)(*[p for p, _ in b]), (C.c_int64 * n)(*[ld for _, ld in b])
    pws, nws = _NO_MATRIX if workspace is None else _workspace(workspace, dev)
    rc = lib().fsdp_newton_schulz(n, rows, cols, pa, la, code, pb, lb, out, steps, _coeffs(coeffs, steps), eps, pws, nws,
                                  _stream(stream, dev))
    if rc:
        _check(rc, "fsdp_newton_schulz")


def fsdp_zero1_muon_workspace_bytes(layout: Layout, tensors) -> int:
    """Scratch bytes of fsdp_zero1_muon_broadcast for these tensors of the layout."""
    ids = (C.c_int32 * max(len(tensors), 1))(*tensors)
    return int(lib().fsdp_zero1_muon_workspace_bytes(layout.handle, len(tensors), ids))


def fsdp_zero1_muon_broadcast(layout: Layout, tensors, grad_replicas, master, momentum, param_replicas,
                              hp: Optional[MuonHparams] = None, workspace=None, coeffs=None, stream=None,
                              grad_dtype: Optional[int] = None, param_dtype: Optional[int] = None) -> None:
    """The ZeRO-1 owner step with Muon for the listed tensors (weight matrices) of a ZeRO-1 layout: mean
    of the N gradient replicas, momentum, Newton-Schulz steps, weight decay, the new weights into
    master and all N replicas.  The layout's other tensors are not touched."""
    if len(grad_replicas) != layout.N or len(param_replicas) != layout.N:
        raise ValueError(f"need {layout.N} gradient and parameter replicas")
    if grad_dtype is None:
        grad_dtype = _dtype_code(grad_replicas[0])
    if param_dtype is None:
        param_dtype = _dtype_code(param_replicas[0])
    hp = MuonHparams() if hp is None else hp
    ids = (C.c_int32 * max(len(tensors), 1))(*tensors)
    pws, nws = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
    _check(lib().fsdp_zero1_muon_broadcast(layout.handle, len(tensors), ids, _ptr_array(grad_replicas), grad_dtype, _ptr(master),
                                           _ptr(momentum), _ptr_array(param_replicas), param_dtype, C.byref(hp),
                                           _coeffs(coeffs, hp.steps), pws, nws, _stream(stream)), "fsdp_zero1_muon_broadcast")


def fsdp_reshard(layout: Layout, unit_begin: int, unit_end: int, full=None, master=None, param_shards=None,
                 stream=None, full_dtype: Optional[int] = None) -> None:
    if full is not None and full_dtype is None:
        full_dtype = _dtype_code(full)
    _check(lib().fsdp_reshard(layout.handle, unit_begin, unit_end, _ptr(full), full_dtype or 0, _ptr(master),
                              _ptr(param_shards), _stream(stream)), "fsdp_reshard")


def fsdp_check_status(stream=None) -> None:
    _check(lib().fsdp_check_status(_stream(stream)), "fsdp_check_status")


def fsdp_set_rs_kernel(kind) -> int:
    """Selects the kernel of fsdp_reduce_scatter_adamw ("auto", "direct", "staged"
    or the FSDP_RS_* code); returns the previous code."""
    code = RS_KERNELS[kind] if isinstance(kind, str) else int(kind)
    prev = lib().fsdp_set_rs_kernel(code)
    if prev < 0:
        raise FsdpError(prev, "fsdp_set_rs_kernel")
    return prev


def fsdp_rs_kernel_for(layout: Layout, grad_dtype) -> str:
    """"direct" or "staged": the kernel fsdp_reduce_scatter_adamw runs for this
    layout and gradient dtype (a torch dtype or FSDP_F32/FSDP_BF16) right now."""
    import torch
    code = grad_dtype if isinstance(grad_dtype, int) else {torch.float32: FSDP_F32, torch.bfloat16: FSDP_BF16}[grad_dtype]
    rc = lib().fsdp_rs_kernel_for(layout.handle, code)
    if rc < 0:
        raise FsdpError(rc, "fsdp_rs_kernel_for")
    return {FSDP_RS_DIRECT: "direct", FSDP_RS_STAGED: "staged"}[rc]


def fsdp_wait_selftest(timeout_ns: int, stream=None) -> None:
    _check(lib().fsdp_wait_selftest(int(timeout_ns), _stream(stream)), "fsdp_wait_selftest")


def fsdp_error_string(status: int) -> str:
    return lib().fsdp_error_string(status).decode()


from .state import ShardedState, StepGraph, step_schedule  # noqa: E402  (harness over the calls above)
from .zero1 import Zero1State  # noqa: E402  (ZeRO-1 state: Muon for matrices, AdamW for the rest)
from .hostfeed import HostFeed  # noqa: E402  (host-fed steps over ShardedState)
from .mlp import ResidualMLP, tensor_views  # noqa: E402  (layers between the all-gather and the reduce-scatter)
