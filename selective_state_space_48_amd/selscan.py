"""Python binding of libselscan (ctypes).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libselscan.so``. PyTorch provides device memory and the current
stream. Importing this module loads the library and fails loudly if it has
not been built (``python -m selective_state_space_48_amd.build``).

Layouts (contiguous): x, delta, z, y ``[batch, dim, L]``; B, C ``[batch, N, L]``;
A ``[dim, N]`` fp32; D, dt_bias ``[dim]`` fp32; states ``[batch, dim, N]`` fp32.
x, delta, z, B, C (and y) share one dtype: float32 or bfloat16.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libselscan.so")

F32, BF16 = 0, 1
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}

# Return codes (include/selscan.h)
OK, ERR_NULL, ERR_DIMS, ERR_DSTATE, ERR_DTYPE, ERR_LAUNCH, ERR_ALLOC, ERR_ALIGN, ERR_ALIAS, \
    ERR_CONFIG, ERR_SCRATCH = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9, -10
# Bytes of the device scratch array behind fwd_noalloc (per GPU)
NOALLOC_SCRATCH_BYTES = 64 << 20


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class FwdOpts(ctypes.Structure):
    _fields_ = [("h0", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64), ("segments", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("ckpt", ctypes.c_void_p),
                ("conv_w", ctypes.c_void_p), ("conv_b", ctypes.c_void_p),
                ("conv_x_prev", ctypes.c_void_p), ("conv_x_last", ctypes.c_void_p),
                ("variant", ctypes.c_int32)]


class StepOpts(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("conv_b", ctypes.c_void_p), ("conv_state", ctypes.c_void_p)]


class BwdOpts(ctypes.Structure):
    _fields_ = [("h0", ctypes.c_void_p), ("dlast_state", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
                ("segments", ctypes.c_int32), ("ckpt", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


class SsdDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class LinattnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class LinattnOpts(ctypes.Structure):
    _fields_ = [("h0", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("segments", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64)]


class LinattnBwdOpts(ctypes.Structure):
    _fields_ = [("h0", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("dlast_state", ctypes.c_void_p),
                ("dh0", ctypes.c_void_p), ("scale", ctypes.c_float), ("segments", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


class GroupnormDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("spatial", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class GroupnormOpts(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


class GatedDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32)]


class GatedOpts(ctypes.Structure):
    _fields_ = [("h0", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("ckpt", ctypes.c_void_p),
                ("segments", ctypes.c_int32), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


class GatedBwdOpts(ctypes.Structure):
    _fields_ = [("h0", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("dlast_state", ctypes.c_void_p),
                ("dh0", ctypes.c_void_p), ("ckpt", ctypes.c_void_p), ("segments", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


class AddnormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32), ("post", ctypes.c_int32),
                ("pre", ctypes.c_int32), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("res_scale", ctypes.c_float)]


class AddnormOpts(ctypes.Structure):
    _fields_ = [("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("pre_bias", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_uint64)]


class AddnormGrads(ctypes.Structure):
    _fields_ = [("dpost_weight", ctypes.c_void_p), ("dpost_bias", ctypes.c_void_p), ("dpre_weight", ctypes.c_void_p),
                ("dpre_bias", ctypes.c_void_p), ("dgate", ctypes.c_void_p)]


class RotaryDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("width", ctypes.c_int64), ("rot", ctypes.c_int64),
                ("offset", ctypes.c_int64), ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("scale", ctypes.c_float)]


class SelscanError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libselscan error {code}: {msg}")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m selective_state_space_48_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fp, i32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32
    dims_p = ctypes.POINTER(Dims)
    lib.selscan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, fp, dims_p, vp]
    lib.selscan_fwd.restype = ctypes.c_int
    opts_p = ctypes.POINTER(FwdOpts)
    lib.selscan_fwd_ex.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, fp, dims_p, opts_p, vp]
    lib.selscan_fwd_ex.restype = ctypes.c_int
    lib.selscan_fwd_noalloc.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, fp, dims_p, vp]
    lib.selscan_fwd_noalloc.restype = ctypes.c_int
    lib.selscan_fwd_workspace_size.argtypes = [dims_p, opts_p, ctypes.POINTER(ctypes.c_uint64)]
    lib.selscan_fwd_workspace_size.restype = ctypes.c_int
    lib.selscan_timing_start.argtypes = [i32]
    lib.selscan_timing_start.restype = ctypes.c_int
    lib.selscan_timing_stop.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i32)]
    lib.selscan_timing_stop.restype = ctypes.c_int
    lib.selscan_step.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp, vp, dims_p, vp]
    lib.selscan_step.restype = ctypes.c_int
    lib.selscan_step_ex.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp, vp, dims_p, ctypes.POINTER(StepOpts), vp]
    lib.selscan_step_ex.restype = ctypes.c_int
    lib.selscan_bwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, vp, vp, fp, vp, vp, fp, vp, fp,
                                dims_p, vp]
    lib.selscan_bwd.restype = ctypes.c_int
    lib.selscan_bwd_ex.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, vp, vp, vp, fp, vp, vp, fp, vp,
                                   fp, dims_p, ctypes.POINTER(BwdOpts), vp]
    lib.selscan_bwd_ex.restype = ctypes.c_int
    lib.selscan_bwd_workspace_size.argtypes = [dims_p, ctypes.POINTER(BwdOpts), ctypes.POINTER(ctypes.c_uint64)]
    lib.selscan_bwd_workspace_size.restype = ctypes.c_int
    lib.selscan_ssd_fwd.argtypes = [vp, vp, fp, vp, vp, fp, fp, vp, fp, ctypes.POINTER(SsdDims), vp]
    lib.selscan_ssd_fwd.restype = ctypes.c_int
    lib.selscan_ssd_fwd_ex.argtypes = [vp, vp, fp, vp, vp, fp, fp, fp, vp, fp, ctypes.POINTER(SsdDims), vp]
    lib.selscan_ssd_fwd_ex.restype = ctypes.c_int
    lib.selscan_ssd_step.argtypes = [fp, vp, vp, fp, vp, vp, fp, fp, vp, ctypes.POINTER(SsdDims), vp]
    lib.selscan_ssd_step.restype = ctypes.c_int
    u64_p = ctypes.POINTER(ctypes.c_uint64)
    la_p, gn_p, gno_p = (ctypes.POINTER(t) for t in (LinattnDims, GroupnormDims, GroupnormOpts))
    la_o, la_bo = ctypes.POINTER(LinattnOpts), ctypes.POINTER(LinattnBwdOpts)
    lib.selscan_linattn_fwd.argtypes = [vp, vp, vp, fp, vp, fp, la_p, la_o, vp]
    lib.selscan_linattn_fwd_workspace_size.argtypes = [la_p, la_o, u64_p]
    lib.selscan_linattn_step.argtypes = [fp, vp, vp, vp, fp, vp, la_p, ctypes.c_float, vp]
    lib.selscan_linattn_bwd.argtypes = [vp, vp, vp, fp, vp, vp, vp, vp, fp, la_p, la_bo, vp]
    lib.selscan_linattn_bwd_workspace_size.argtypes = [la_p, la_bo, i32, u64_p]
    lib.selscan_groupnorm.argtypes = [vp, fp, fp, vp, vp, fp, fp, gn_p, gno_p, vp]
    lib.selscan_groupnorm_bwd.argtypes = [vp, fp, fp, vp, vp, fp, fp, vp, fp, fp, vp, gn_p, gno_p, vp]
    lib.selscan_groupnorm_workspace_size.argtypes = [gn_p, i32, u64_p]
    for f in (lib.selscan_linattn_fwd, lib.selscan_linattn_fwd_workspace_size, lib.selscan_linattn_step,
              lib.selscan_linattn_bwd, lib.selscan_linattn_bwd_workspace_size, lib.selscan_groupnorm,
              lib.selscan_groupnorm_bwd, lib.selscan_groupnorm_workspace_size):
        f.restype = ctypes.c_int
    ga_p, ga_o, ga_bo = (ctypes.POINTER(t) for t in (GatedDims, GatedOpts, GatedBwdOpts))
    an_p, an_o, an_g = (ctypes.POINTER(t) for t in (AddnormDims, AddnormOpts, AddnormGrads))
    lib.selscan_gated_fwd.argtypes = [vp, vp, vp, fp, vp, vp, fp, ga_p, ga_o, vp]
    lib.selscan_gated_fwd_workspace_size.argtypes = [ga_p, ga_o, u64_p]
    lib.selscan_gated_step.argtypes = [fp, vp, vp, vp, fp, vp, vp, ga_p, vp]
    lib.selscan_gated_bwd.argtypes = [vp, vp, vp, fp, vp, vp, vp, vp, vp, fp, vp, ga_p, ga_bo, vp]
    lib.selscan_gated_bwd_workspace_size.argtypes = [ga_p, ga_bo, u64_p]
    lib.selscan_addnorm.argtypes = [vp, vp, vp, vp, fp, an_p, an_o, vp]
    lib.selscan_addnorm_bwd.argtypes = [vp, vp, fp, vp, vp, vp, vp, an_g, an_p, an_o, vp]
    lib.selscan_addnorm_bwd_workspace_size.argtypes = [an_p, an_o, an_g, u64_p]
    lib.selscan_rotary.argtypes = [vp, vp, fp, vp, vp, vp, ctypes.POINTER(RotaryDims), vp]
    for name in ("gated_fwd", "gated_fwd_workspace_size", "gated_step", "gated_bwd", "gated_bwd_workspace_size",
                 "addnorm", "addnorm_bwd", "addnorm_bwd_workspace_size", "rotary"):
        getattr(lib, "selscan_" + name).restype = ctypes.c_int
    lib.selscan_conv1d.argtypes = [vp, fp, fp, fp, vp, fp, dims_p, vp]
    lib.selscan_conv1d.restype = ctypes.c_int
    lib.selscan_conv1d_step.argtypes = [fp, vp, fp, fp, vp, dims_p, vp]
    lib.selscan_conv1d_bwd.argtypes = [vp, fp, fp, fp, vp, vp, fp, fp, fp, dims_p, vp]
    lib.selscan_conv1d_bwd.restype = ctypes.c_int
    lib.selscan_conv1d_step.restype = ctypes.c_int
    lib.selscan_strerror.argtypes = [ctypes.c_int]
    lib.selscan_strerror.restype = ctypes.c_char_p
    lib.selscan_version.argtypes = []
    lib.selscan_version.restype = ctypes.c_int
    return lib


lib = _load()


def version() -> int:
    return lib.selscan_version()


def strerror(code: int) -> str:
    return lib.selscan_strerror(code).decode()


def _check(code: int) -> None:
    if code != OK:
        raise SelscanError(code, strerror(code))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _req(t: Optional[torch.Tensor], name: str, dtype=None, shape=None, device=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The current stream's handle without a Stream object around it (0.1 instead of
# 2 us a call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def workspace_size(batch: int, L: int, dim: int, dtype: torch.dtype, N: int = 16, *,
                   segments: int = 0, groups: int = 0, ckpt: bool = False,
                   conv: bool = False, variant: int = 0) -> int:
    """Bytes of device workspace a forward call of this shape needs; ``ckpt`` and
    ``conv`` say whether the call passes checkpoints or the fused convolution's
    taps (they restrict the automatic plan to 4-wave launches)."""
    dims = Dims(batch, L, dim, N, _DTYPES[dtype])
    # The size query looks only at whether these options are set, never at
    # the memory: a placeholder address stands for "set".
    flag = ctypes.c_void_p(256)
    opts = FwdOpts(None, None, 0, int(segments), int(groups), flag if ckpt else None,
                   flag if conv else None, None, None, None, int(variant))
    out = ctypes.c_uint64(0)
    _check(lib.selscan_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(out)))
    return int(out.value)


def bwd_workspace_size(batch: int, L: int, dim: int, dtype: torch.dtype, N: int = 16, *,
                       segments: int = 0, ckpt: bool = False) -> int:
    """Bytes of device workspace a backward call of this shape needs (``ckpt``:
    the call is given the forward's checkpoints)."""
    dims = Dims(batch, L, dim, N, _DTYPES[dtype])
    opts = BwdOpts(None, None, None, int(segments), ctypes.c_void_p(256) if ckpt else None)
    out = ctypes.c_uint64(0)
    _check(lib.selscan_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(out)))
    return int(out.value)


def timing_start(capacity: int) -> None:
    """Record HIP events around the next ``capacity`` output-pass / step kernels."""
    _check(lib.selscan_timing_start(int(capacity)))


def timing_stop() -> Tuple[float, int]:
    """Wait for the recorded kernels; return (summed milliseconds, launches)."""
    ms, n = ctypes.c_double(0.0), ctypes.c_int32(0)
    _check(lib.selscan_timing_stop(ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


def ckpt_shape(batch: int, dim: int, L: int, N: int = 16) -> Tuple[int, int, int, int]:
    """Shape of the forward's checkpoints: the state before every 16th token."""
    return ((L + 15) // 16, batch, dim, N)


def fwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
        D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
        dt_bias: Optional[torch.Tensor] = None, *, y: Optional[torch.Tensor] = None,
        last_state: Optional[torch.Tensor] = None, return_last_state: bool = True,
        h0: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
        segments: int = 0, groups: int = 0, variant: int = 0,
        ckpt: Optional[torch.Tensor] = None, conv_w: Optional[torch.Tensor] = None,
        conv_b: Optional[torch.Tensor] = None, conv_x_prev: Optional[torch.Tensor] = None,
        conv_x_last: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective-scan forward (selscan_fwd_ex). Returns (y, last_state).

    ``ckpt`` (shape ``ckpt_shape(batch, dim, L)``, fp32) receives the state
    entering every 16th token, for ``bwd(..., ckpt=ckpt)``. With ``conv_w``
    [dim, 4] fp32 the block's causal conv1d + SiLU (as ``conv1d``) is applied
    to ``x`` inside the scan; ``conv_b`` [dim], ``conv_x_prev`` and
    ``conv_x_last`` [batch, dim, 3] fp32 as for ``conv1d``.

    ``y`` and ``last_state`` may be passed in preallocated; otherwise they are
    allocated here. ``h0`` [batch, dim, N] fp32 is the state entering token 0
    (None: zeros; it may be ``last_state`` itself). ``workspace`` is a uint8
    device tensor of at least ``workspace_size(...)`` bytes; by default one is
    taken from torch's caching allocator. ``segments``/``groups``/``variant``
    select the launch (0 = automatic; see selscan_fwd_opts_t).
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    batch, dim, L = x.shape
    dev = x.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    N = A.shape[-1] if A.dim() == 2 else -1
    _req(x, "x", x.dtype, (batch, dim, L), dev)
    _req(delta, "delta", x.dtype, (batch, dim, L), dev)
    _req(z, "z", x.dtype, (batch, dim, L), dev)
    _req(A, "A", torch.float32, (dim, N), dev)
    _req(B, "B", x.dtype, (batch, N, L), dev)
    _req(C, "C", x.dtype, (batch, N, L), dev)
    _req(D, "D", torch.float32, (dim,), dev)
    _req(dt_bias, "dt_bias", torch.float32, (dim,), dev)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", x.dtype, (batch, dim, L), dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    _req(last_state, "last_state", torch.float32, (batch, dim, N), dev)
    _req(h0, "h0", torch.float32, (batch, dim, N), dev)
    _req(ckpt, "ckpt", torch.float32, ckpt_shape(batch, dim, L, N), dev)
    _req(conv_w, "conv_w", torch.float32, (dim, CONV_WIDTH), dev)
    _req(conv_b, "conv_b", torch.float32, (dim,), dev)
    _req(conv_x_prev, "conv_x_prev", torch.float32, (batch, dim, CONV_WIDTH - 1), dev)
    _req(conv_x_last, "conv_x_last", torch.float32, (batch, dim, CONV_WIDTH - 1), dev)
    dims = Dims(batch, L, dim, N, _DTYPES[x.dtype])
    opts = FwdOpts(None, None, 0, int(segments), int(groups), _ptr(ckpt), _ptr(conv_w), _ptr(conv_b),
                   _ptr(conv_x_prev), _ptr(conv_x_last), int(variant))
    need = ctypes.c_uint64(0)
    _check(lib.selscan_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(need)))
    if workspace is None and need.value > 0:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, None, dev)
        opts.workspace = workspace.data_ptr()
        opts.workspace_bytes = workspace.numel()
    if h0 is not None:
        opts.h0 = h0.data_ptr()
    rc = lib.selscan_fwd_ex(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                            _ptr(dt_bias), _ptr(y), _ptr(last_state), ctypes.byref(dims),
                            ctypes.byref(opts), _stream(dev))
    _check(rc)
    return y, last_state


def fwd_noalloc(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                dt_bias: Optional[torch.Tensor] = None, *, y: torch.Tensor,
                last_state: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """selscan_fwd_noalloc: the forward with its workspace in the library's
    static device scratch (NOALLOC_SCRATCH_BYTES per GPU) instead of an
    allocation. ``y`` (and ``last_state``, if wanted) must be passed in: this
    call allocates nothing, here or in the library. Calls that overlap in time
    on one GPU share the scratch and must not be made."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    batch, dim, L = x.shape
    dev = x.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    N = A.shape[-1] if A.dim() == 2 else -1
    for t, name, dt, shape in ((x, "x", x.dtype, (batch, dim, L)), (delta, "delta", x.dtype, (batch, dim, L)),
                               (z, "z", x.dtype, (batch, dim, L)), (A, "A", torch.float32, (dim, N)),
                               (B, "B", x.dtype, (batch, N, L)), (C, "C", x.dtype, (batch, N, L)),
                               (D, "D", torch.float32, (dim,)), (dt_bias, "dt_bias", torch.float32, (dim,)),
                               (y, "y", x.dtype, (batch, dim, L)),
                               (last_state, "last_state", torch.float32, (batch, dim, N))):
        _req(t, name, dt, shape, dev)
    dims = Dims(batch, L, dim, N, _DTYPES[x.dtype])
    rc = lib.selscan_fwd_noalloc(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                 _ptr(dt_bias), _ptr(y), _ptr(last_state), ctypes.byref(dims), _stream(dev))
    _check(rc)
    return y, last_state


def step(state: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
         B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor] = None,
         z: Optional[torch.Tensor] = None, *, y: Optional[torch.Tensor] = None,
         conv_w: Optional[torch.Tensor] = None, conv_b: Optional[torch.Tensor] = None,
         conv_state: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step (selscan_step / selscan_step_ex): updates ``state`` in place and
    returns y [batch, dim].

    ``delta`` is the pre-activation with any channel bias already added. With
    ``conv_w`` [dim, 4] (and ``conv_b`` [dim], ``conv_state`` [batch, dim, 3]
    fp32, shifted in place) the block's convolution + SiLU is applied to x
    first, in the same kernel.
    """
    if state.dim() != 3:
        raise ValueError("state must be [batch, dim, N]")
    batch, dim, N = state.shape
    dev = state.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    _req(state, "state", torch.float32, (batch, dim, N), dev)
    _req(x, "x", x.dtype, (batch, dim), dev)
    _req(delta, "delta", x.dtype, (batch, dim), dev)
    _req(z, "z", x.dtype, (batch, dim), dev)
    _req(A, "A", torch.float32, (dim, N), dev)
    _req(B, "B", x.dtype, (batch, N), dev)
    _req(C, "C", x.dtype, (batch, N), dev)
    _req(D, "D", torch.float32, (dim,), dev)
    _req(conv_w, "conv_w", torch.float32, (dim, CONV_WIDTH), dev)
    _req(conv_b, "conv_b", torch.float32, (dim,), dev)
    _req(conv_state, "conv_state", torch.float32, (batch, dim, CONV_WIDTH - 1), dev)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", x.dtype, (batch, dim), dev)
    dims = Dims(batch, 1, dim, N, _DTYPES[x.dtype])
    if conv_w is None and conv_b is None and conv_state is None:
        rc = lib.selscan_step(_ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                              _ptr(z), _ptr(y), ctypes.byref(dims), _stream(dev))
    else:
        opts = StepOpts(_ptr(conv_w), _ptr(conv_b), _ptr(conv_state))
        rc = lib.selscan_step_ex(_ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                 _ptr(z), _ptr(y), ctypes.byref(dims), ctypes.byref(opts), _stream(dev))
    _check(rc)
    return y


def bwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
        D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
        dt_bias: Optional[torch.Tensor] = None, *, dy: torch.Tensor,
        want_dD: bool = True, want_ddt_bias: bool = True, segments: int = 0,
        h0: Optional[torch.Tensor] = None, dlast_state: Optional[torch.Tensor] = None,
        want_dh0: bool = False, ckpt: Optional[torch.Tensor] = None,
        workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass (selscan_bwd): gradients for the output gradient ``dy``.

    Returns a dict with dx, ddelta, dB, dC (input dtype), dA [dim, N] fp32, and
    dz (when z is given), dD and ddt_bias ([dim] fp32, when wanted).
    ``h0`` (the forward's initial state), ``dlast_state`` (the gradient into
    its final state), ``want_dh0`` (adds dh0 [batch, dim, N] fp32), ``ckpt``
    (the checkpoints a ``fwd(..., ckpt=...)`` over the same inputs wrote) and
    ``segments`` other than 0 (automatic) are passed to selscan_bwd_ex.
    ``workspace`` is a uint8 device tensor of at least ``bwd_workspace_size(...)``
    bytes; by default one is taken from torch's allocator, so that the library
    allocates nothing.
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    batch, dim, L = x.shape
    dev = x.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    N = A.shape[-1] if A.dim() == 2 else -1
    for t, name, dt, shape in ((x, "x", x.dtype, (batch, dim, L)), (delta, "delta", x.dtype, (batch, dim, L)),
                               (z, "z", x.dtype, (batch, dim, L)), (dy, "dy", x.dtype, (batch, dim, L)),
                               (A, "A", torch.float32, (dim, N)), (B, "B", x.dtype, (batch, N, L)),
                               (C, "C", x.dtype, (batch, N, L)), (D, "D", torch.float32, (dim,)),
                               (dt_bias, "dt_bias", torch.float32, (dim,)),
                               (h0, "h0", torch.float32, (batch, dim, N)),
                               (dlast_state, "dlast_state", torch.float32, (batch, dim, N)),
                               (ckpt, "ckpt", torch.float32, ckpt_shape(batch, dim, L, N))):
        _req(t, name, dt, shape, dev)
    out = {"dx": torch.empty_like(x), "ddelta": torch.empty_like(x), "dB": torch.empty_like(B),
           "dC": torch.empty_like(C), "dA": torch.empty_like(A)}
    if z is not None:
        out["dz"] = torch.empty_like(x)
    if want_dD:
        out["dD"] = torch.empty((dim,), dtype=torch.float32, device=dev)
    if want_ddt_bias:
        out["ddt_bias"] = torch.empty((dim,), dtype=torch.float32, device=dev)
    if want_dh0:
        out["dh0"] = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    dims = Dims(batch, L, dim, N, _DTYPES[x.dtype])
    args = (_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias),
            _ptr(dy), _ptr(out["dx"]), _ptr(out["ddelta"]), _ptr(out["dA"]), _ptr(out["dB"]),
            _ptr(out["dC"]), _ptr(out.get("dD")), _ptr(out.get("dz")), _ptr(out.get("ddt_bias")),
            ctypes.byref(dims))
    opts = BwdOpts(_ptr(h0), _ptr(dlast_state), _ptr(out.get("dh0")), segments, _ptr(ckpt))
    need = ctypes.c_uint64(0)
    _check(lib.selscan_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(need)))
    if workspace is None and need.value > 0:
        workspace = torch.empty(int(need.value), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, None, dev)
        opts.workspace = workspace.data_ptr()
        opts.workspace_bytes = workspace.numel()
    _check(lib.selscan_bwd_ex(*args, ctypes.byref(opts), _stream(dev)))
    return out


def ssd_fwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
            C: torch.Tensor, D: Optional[torch.Tensor] = None,
            dt_bias: Optional[torch.Tensor] = None, *, y: Optional[torch.Tensor] = None,
            last_state: Optional[torch.Tensor] = None, return_last_state: bool = True,
            h0: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Mamba-2 SSD layer (selscan_ssd_fwd), bfloat16. Returns (y, last_state).

    ``x`` [batch, L, heads, 64]; ``delta`` [batch, L, heads] (before softplus);
    ``A``, ``D``, ``dt_bias`` [heads] fp32; ``B``, ``C`` [batch, L, dstate];
    last_state [batch, heads, dstate, 64] fp32. ``h0`` (same shape) is the
    state entering token 0 (selscan_ssd_fwd_ex; None: zeros).
    """
    if x.dim() != 4:
        raise ValueError("x must be [batch, L, heads, headdim]")
    batch, L, H, P = x.shape
    N = B.shape[-1] if B.dim() == 3 else -1
    dev = x.device
    bf = torch.bfloat16
    _req(x, "x", bf, (batch, L, H, P), dev)
    _req(delta, "delta", bf, (batch, L, H), dev)
    _req(A, "A", torch.float32, (H,), dev)
    _req(B, "B", bf, (batch, L, N), dev)
    _req(C, "C", bf, (batch, L, N), dev)
    _req(D, "D", torch.float32, (H,), dev)
    _req(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", bf, (batch, L, H, P), dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, H, N, P), dtype=torch.float32, device=dev)
    _req(last_state, "last_state", torch.float32, (batch, H, N, P), dev)
    _req(h0, "h0", torch.float32, (batch, H, N, P), dev)
    dims = SsdDims(batch, L, H, P, N, BF16)
    if h0 is None:
        _check(lib.selscan_ssd_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                   _ptr(dt_bias), _ptr(y), _ptr(last_state), ctypes.byref(dims),
                                   _stream(dev)))
    else:
        _check(lib.selscan_ssd_fwd_ex(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                      _ptr(dt_bias), _ptr(h0), _ptr(y), _ptr(last_state),
                                      ctypes.byref(dims), _stream(dev)))
    return y, last_state


def ssd_step(state: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
             B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor] = None,
             dt_bias: Optional[torch.Tensor] = None, *,
             y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step of the SSD layer (selscan_ssd_step): updates ``state``
    [batch, heads, dstate, 64] fp32 in place and returns y [batch, heads, 64].
    ``x`` [batch, heads, 64], ``delta`` [batch, heads], ``B``, ``C`` [batch,
    dstate] bf16; ``A``, ``D``, ``dt_bias`` [heads] fp32."""
    if state.dim() != 4:
        raise ValueError("state must be [batch, heads, dstate, headdim]")
    batch, H, N, P = state.shape
    dev = state.device
    bf = torch.bfloat16
    _req(state, "state", torch.float32, (batch, H, N, P), dev)
    _req(x, "x", bf, (batch, H, P), dev)
    _req(delta, "delta", bf, (batch, H), dev)
    _req(A, "A", torch.float32, (H,), dev)
    _req(B, "B", bf, (batch, N), dev)
    _req(C, "C", bf, (batch, N), dev)
    _req(D, "D", torch.float32, (H,), dev)
    _req(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", bf, (batch, H, P), dev)
    dims = SsdDims(batch, 1, H, P, N, BF16)
    _check(lib.selscan_ssd_step(_ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
                                _ptr(D), _ptr(dt_bias), _ptr(y), ctypes.byref(dims), _stream(dev)))
    return y


_HERE = contextlib.nullcontext()


def _device(dev: torch.device):
    """The device the call launches on, made current where it is not."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {dev}")
    return torch.cuda.device(dev) if dev.index != torch.cuda.current_device() else _HERE


def _scratch(workspace: Optional[torch.Tensor], need: int, dev: torch.device) -> Optional[torch.Tensor]:
    """The caller's workspace, checked, or one of ``need`` bytes from torch's allocator (None for 0)."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    _req(workspace, "workspace", torch.uint8, None, dev)
    return workspace


def _scale(scale: Optional[float]) -> float:
    """The C calls' scale: 0 stands for 1 / sqrt(dk)."""
    if scale is None:
        return 0.0
    if ctypes.c_float(scale).value == 0:  # (a double that fp32 has no number for, too)
        raise ValueError("scale must not be 0 in fp32 (None: 1 / sqrt(dk))")
    return float(scale)


def _linattn_dims(q, k, v, L, dtype) -> "LinattnDims":
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    return LinattnDims(q.shape[0], L, q.shape[-2], k.shape[-2], q.shape[-1], v.shape[-1], _DTYPES[dtype])


def linattn_workspace_size(batch: int, L: int, heads: int, kv_heads: int, dk: int, dv: int, dtype: torch.dtype, *,
                           segments: int = 0) -> int:
    """Bytes of device workspace a ``linattn_fwd`` call of this shape needs."""
    dims = LinattnDims(batch, L, heads, kv_heads, dk, dv, _DTYPES[dtype])
    opts = LinattnOpts(None, None, 0.0, int(segments), None, 0)
    out = ctypes.c_uint64(0)
    _check(lib.selscan_linattn_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(out)))
    return int(out.value)


def linattn_bwd_workspace_size(batch: int, L: int, heads: int, kv_heads: int, dk: int, dv: int, dtype: torch.dtype,
                               *, segments: int = 0, want_dlog_decay: bool = True) -> int:
    """Bytes of device workspace a ``linattn_bwd`` call of this shape needs."""
    dims = LinattnDims(batch, L, heads, kv_heads, dk, dv, _DTYPES[dtype])
    opts = LinattnBwdOpts(None, None, None, None, 0.0, int(segments), None, 0)
    out = ctypes.c_uint64(0)
    _check(lib.selscan_linattn_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), int(want_dlog_decay),
                                                  ctypes.byref(out)))
    return int(out.value)


def linattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                scale: Optional[float] = None, h0: Optional[torch.Tensor] = None,
                lengths: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                last_state: Optional[torch.Tensor] = None, return_last_state: bool = True, segments: int = 0,
                workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay for each head (selscan_linattn_fwd). Returns (y, last_state).

    ``q`` [batch, L, heads, dk]; ``k``, ``v`` [batch, L, kv_heads, dk / dv]
    (heads a multiple of kv_heads; float32 or bfloat16); ``log_decay`` [heads]
    fp32, the logarithm of each head's decay per token; y [batch, L, heads, dv],
    last_state [batch, heads, dk, dv] fp32. ``h0`` (same shape) is the state
    entering token 0 (it may be ``last_state`` itself); ``lengths`` [batch]
    int32 the tokens of each entry (y is 0 behind them); ``scale`` multiplies q
    (None: 1 / sqrt(dk)). ``segments`` and ``workspace`` as for ``fwd``
    (``linattn_workspace_size``).
    """
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [batch, L, heads, width]")
    batch, L, H, dk = q.shape
    Hk, dv = k.shape[2], v.shape[3]
    dev, dt = q.device, q.dtype
    dims = _linattn_dims(q, k, v, L, dt)
    _req(q, "q", dt, None, dev)
    _req(k, "k", dt, (batch, L, Hk, dk), dev)
    _req(v, "v", dt, (batch, L, Hk, dv), dev)
    _req(log_decay, "log_decay", torch.float32, (H,), dev)
    _req(h0, "h0", torch.float32, (batch, H, dk, dv), dev)
    _req(lengths, "lengths", torch.int32, (batch,), dev)
    with _device(dev):
        if y is None:
            y = torch.empty((batch, L, H, dv), dtype=dt, device=dev)
        _req(y, "y", dt, (batch, L, H, dv), dev)
        if last_state is None and return_last_state:
            last_state = torch.empty((batch, H, dk, dv), dtype=torch.float32, device=dev)
        _req(last_state, "last_state", torch.float32, (batch, H, dk, dv), dev)
        opts = LinattnOpts(_ptr(h0), _ptr(lengths), _scale(scale), int(segments), None, 0)
        need = ctypes.c_uint64(0)
        _check(lib.selscan_linattn_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(need)))
        workspace = _scratch(workspace, int(need.value), dev)
        if workspace is not None:
            opts.workspace, opts.workspace_bytes = workspace.data_ptr(), workspace.numel()
        _check(lib.selscan_linattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(y), _ptr(last_state),
                                       ctypes.byref(dims), ctypes.byref(opts), _stream(dev)))
    return y, last_state


def linattn_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                 scale: Optional[float] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the layer (selscan_linattn_step): updates ``state`` [batch,
    heads, dk, dv] fp32 in place and returns y [batch, heads, dv]. ``q`` [batch,
    heads, dk]; ``k``, ``v`` [batch, kv_heads, dk / dv]; ``log_decay`` [heads]
    fp32; ``scale`` as for ``linattn_fwd``."""
    if state.dim() != 4 or q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("state must be [batch, heads, dk, dv] and q, k, v [batch, heads, width]")
    batch, H, dk, dv = state.shape
    dev, dt, Hk = state.device, q.dtype, k.shape[1]
    _req(state, "state", torch.float32, (batch, H, dk, dv), dev)
    _req(q, "q", dt, (batch, H, dk), dev)
    _req(k, "k", dt, (batch, Hk, dk), dev)
    _req(v, "v", dt, (batch, Hk, dv), dev)
    _req(log_decay, "log_decay", torch.float32, (H,), dev)
    dims = _linattn_dims(q, k, v, 1, dt)
    with _device(dev):
        if y is None:
            y = torch.empty((batch, H, dv), dtype=dt, device=dev)
        _req(y, "y", dt, (batch, H, dv), dev)
        _check(lib.selscan_linattn_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(y),
                                        ctypes.byref(dims), _scale(scale), _stream(dev)))
    return y


def linattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *, dy: torch.Tensor,
                scale: Optional[float] = None, h0: Optional[torch.Tensor] = None,
                lengths: Optional[torch.Tensor] = None, dlast_state: Optional[torch.Tensor] = None,
                want_dlog_decay: bool = True, want_dh0: bool = False, segments: int = 0,
                workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``linattn_fwd`` (selscan_linattn_bwd) for ``dy`` [batch, L,
    heads, dv] and, when given, ``dlast_state`` (the gradient into last_state).

    Returns a dict with dq, dk, dv (like q, k, v; 0 behind an entry's length),
    dlog_decay [heads] fp32 and dh0 [batch, heads, dk, dv] fp32 when wanted.
    ``workspace``: at least ``linattn_bwd_workspace_size(...)`` bytes.
    """
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [batch, L, heads, width]")
    batch, L, H, dk = q.shape
    Hk, dv = k.shape[2], v.shape[3]
    dev, dt = q.device, q.dtype
    dims = _linattn_dims(q, k, v, L, dt)
    state = (batch, H, dk, dv)
    for t, name, tt, shape in ((q, "q", dt, None), (k, "k", dt, (batch, L, Hk, dk)), (v, "v", dt, (batch, L, Hk, dv)),
                               (dy, "dy", dt, (batch, L, H, dv)), (log_decay, "log_decay", torch.float32, (H,)),
                               (h0, "h0", torch.float32, state), (dlast_state, "dlast_state", torch.float32, state),
                               (lengths, "lengths", torch.int32, (batch,))):
        _req(t, name, tt, shape, dev)
    with _device(dev):
        out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
        if want_dlog_decay:
            out["dlog_decay"] = torch.empty_like(log_decay)
        if want_dh0:
            out["dh0"] = torch.empty(state, dtype=torch.float32, device=dev)
        opts = LinattnBwdOpts(_ptr(h0), _ptr(lengths), _ptr(dlast_state), _ptr(out.get("dh0")), _scale(scale),
                              int(segments), None, 0)
        need = ctypes.c_uint64(0)
        _check(lib.selscan_linattn_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), int(want_dlog_decay),
                                                      ctypes.byref(need)))
        workspace = _scratch(workspace, int(need.value), dev)
        if workspace is not None:
            opts.workspace, opts.workspace_bytes = workspace.data_ptr(), workspace.numel()
        _check(lib.selscan_linattn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(dy), _ptr(out["dq"]),
                                       _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out.get("dlog_decay")),
                                       ctypes.byref(dims), ctypes.byref(opts), _stream(dev)))
    return out


ACTS = {"none": 0, "silu": 1, "gate": 2}


def _groupnorm_dims(x: torch.Tensor, groups: int, act: str, eps: float) -> "GroupnormDims":
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, channels] or [batch, spatial, channels]")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    spatial = x.shape[1] if x.dim() == 3 else 1
    return GroupnormDims(x.shape[0], spatial, x.shape[-1], int(groups), _DTYPES[x.dtype], ACTS[act], float(eps))


def _groupnorm_workspace(dims, backward: bool, workspace, dev) -> Tuple[Optional[torch.Tensor], "GroupnormOpts"]:
    need = ctypes.c_uint64(0)
    _check(lib.selscan_groupnorm_workspace_size(ctypes.byref(dims), int(backward), ctypes.byref(need)))
    workspace = _scratch(workspace, int(need.value), dev)
    return workspace, GroupnormOpts(None, 0) if workspace is None else GroupnormOpts(workspace.data_ptr(),
                                                                                     workspace.numel())


def groupnorm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
              bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, *, act: str = "none",
              eps: float = 1e-5, y: Optional[torch.Tensor] = None, return_stats: bool = True,
              workspace: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Group norm with an activation, channels last (selscan_groupnorm). Returns (y, mean, rstd).

    ``x`` [rows, channels] (each row by itself) or [batch, spatial, channels]
    (over all positions of an entry), float32 or bfloat16; ``weight``, ``bias``
    [channels] fp32. ``act``: "none", "silu" (of the normed value) or "gate"
    (times silu(z), ``z`` like x). mean and rstd [rows, groups] fp32 are what
    ``groupnorm_bwd`` needs (None with ``return_stats=False``).
    """
    dims = _groupnorm_dims(x, groups, act, eps)
    dev, dt, C = x.device, x.dtype, x.shape[-1]
    _req(x, "x", dt, None, dev)
    _req(weight, "weight", torch.float32, (C,), dev)
    _req(bias, "bias", torch.float32, (C,), dev)
    if (z is None) != (act != "gate"):
        raise ValueError('z belongs to act="gate", and to it alone')
    _req(z, "z", dt, x.shape, dev)
    with _device(dev):
        if y is None:
            y = torch.empty_like(x)
        _req(y, "y", dt, x.shape, dev)
        mean = rstd = None
        if return_stats:
            mean, rstd = (torch.empty((x.shape[0], int(groups)), dtype=torch.float32, device=dev) for _ in range(2))
        workspace, opts = _groupnorm_workspace(dims, False, workspace, dev)
        _check(lib.selscan_groupnorm(_ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ptr(y), _ptr(mean), _ptr(rstd),
                                     ctypes.byref(dims), ctypes.byref(opts), _stream(dev)))
    return y, mean, rstd


def groupnorm_bwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, *, act: str = "none",
                  dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, want_dweight: bool = True,
                  want_dbias: bool = True, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``groupnorm`` (selscan_groupnorm_bwd) for ``dy``, from the
    ``mean`` and ``rstd`` that it returned: a dict with dx (like x), dweight and
    dbias [channels] fp32 when wanted, and dz (like z) with the gate."""
    dims = _groupnorm_dims(x, groups, act, 0.0)
    dev, dt, C = x.device, x.dtype, x.shape[-1]
    stats = (x.shape[0], int(groups))
    if (z is None) != (act != "gate"):
        raise ValueError('z belongs to act="gate", and to it alone')
    for t, name, tt, shape in ((x, "x", dt, None), (weight, "weight", torch.float32, (C,)),
                               (bias, "bias", torch.float32, (C,)), (z, "z", dt, x.shape), (dy, "dy", dt, x.shape),
                               (mean, "mean", torch.float32, stats), (rstd, "rstd", torch.float32, stats)):
        _req(t, name, tt, shape, dev)
    with _device(dev):
        out = {"dx": torch.empty_like(x)}
        if want_dweight:
            out["dweight"] = torch.empty((C,), dtype=torch.float32, device=dev)
        if want_dbias:
            out["dbias"] = torch.empty((C,), dtype=torch.float32, device=dev)
        if z is not None:
            out["dz"] = torch.empty_like(z)
        workspace, opts = _groupnorm_workspace(dims, True, workspace, dev)
        _check(lib.selscan_groupnorm_bwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ptr(dy), _ptr(mean),
                                         _ptr(rstd), _ptr(out["dx"]), _ptr(out.get("dweight")),
                                         _ptr(out.get("dbias")), _ptr(out.get("dz")), ctypes.byref(dims),
                                         ctypes.byref(opts), _stream(dev)))
    return out


GATED_MIX, GATED_DECAY = 0, 1
# Tokens between the checkpoints of gated_fwd
GATED_CKPT = 64


def gated_ckpt_shape(batch: int, L: int, dim: int) -> Tuple[int, int, int]:
    """Shape of the checkpoints ``gated_fwd`` writes and ``gated_bwd`` reads."""
    return ((L + GATED_CKPT - 1) // GATED_CKPT, batch, dim)


def _gated_args(x, g, r, A, z, shape, **others) -> "GatedDims":
    """The inputs of the three gated calls, checked; ``others`` are further tensors of x's type and shape."""
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if (r is None) != (A is None):
        raise ValueError("r and A belong together")
    dev = x.device
    _req(x, "x", x.dtype, shape, dev)
    for name, t in dict(g=g, r=r, z=z, **others).items():
        _req(t, name, x.dtype, shape, dev)
    _req(A, "A", torch.float32, (shape[-1],), dev)
    L = shape[1] if len(shape) == 3 else 1
    return GatedDims(shape[0], L, shape[-1], _DTYPES[x.dtype], GATED_MIX if r is None else GATED_DECAY)


# (The sizes alone decide: a call of the same sizes as one before saves the query.)
@functools.lru_cache(maxsize=256)
def _gated_need(batch: int, L: int, dim: int, dtype: int, kind: int, segments: int, backward: bool, ckpt: bool) -> int:
    dims, n = GatedDims(batch, L, dim, dtype, kind), ctypes.c_uint64(0)
    if backward:
        opts = GatedBwdOpts(ckpt=16 if ckpt else None, segments=segments)
        _check(lib.selscan_gated_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(opts), ctypes.byref(n)))
    else:
        _check(lib.selscan_gated_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(GatedOpts(segments=segments)),
                                                    ctypes.byref(n)))
    return int(n.value)


def gated_workspace_size(batch: int, L: int, dim: int, dtype: torch.dtype, *, decay: bool = True,
                         segments: int = 0) -> int:
    """Bytes of workspace ``gated_fwd`` needs for this shape and number of segments."""
    return _gated_need(batch, L, dim, _DTYPES[dtype], int(decay), int(segments), False, False)


def gated_bwd_workspace_size(batch: int, L: int, dim: int, dtype: torch.dtype, *, decay: bool = True,
                             ckpt_given: bool = False, segments: int = 0) -> int:
    """Bytes of workspace ``gated_bwd`` needs for this shape and these choices."""
    return _gated_need(batch, L, dim, _DTYPES[dtype], int(decay), int(segments), True, bool(ckpt_given))


def gated_fwd(x: torch.Tensor, g: torch.Tensor, r: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
              z: Optional[torch.Tensor] = None, *, h0: Optional[torch.Tensor] = None,
              lengths: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
              last_state: Optional[torch.Tensor] = None, return_last_state: bool = True,
              ckpt: Optional[torch.Tensor] = None, segments: int = 0, workspace: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence (selscan_gated_fwd). Returns (y, last_state).

    ``x``, ``g``, ``r``, ``z`` [batch, L, dim] (float32 or bfloat16). Without
    ``r``: h = (1 - u) h + u x, u = sigmoid(g). With ``r`` and ``A`` [dim] fp32
    (at most 0): a = exp(A sigmoid(r)), h = a h + sqrt(1 - a^2) sigmoid(g) x.
    y = h, or h silu(z). ``h0`` [batch, dim] fp32 is the state entering token 0
    (it may be ``last_state`` itself); ``lengths`` [batch] int32 the tokens of
    each entry (y is 0 behind them). ``ckpt`` (``gated_ckpt_shape``) fp32
    receives states for ``gated_bwd``. ``segments`` and ``workspace`` as for
    ``fwd`` (``gated_workspace_size``).
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, dim]")
    batch, L, dim = x.shape
    dev, dt = x.device, x.dtype
    dims = _gated_args(x, g, r, A, z, x.shape)
    _req(h0, "h0", torch.float32, (batch, dim), dev)
    _req(lengths, "lengths", torch.int32, (batch,), dev)
    _req(ckpt, "ckpt", torch.float32, gated_ckpt_shape(batch, L, dim), dev)
    with _device(dev):
        if y is None:
            y = torch.empty_like(x)
        else:
            _req(y, "y", dt, x.shape, dev)
        if last_state is not None:
            _req(last_state, "last_state", torch.float32, (batch, dim), dev)
        elif return_last_state:
            last_state = torch.empty((batch, dim), dtype=torch.float32, device=dev)
        opts = GatedOpts(_ptr(h0), _ptr(lengths), _ptr(ckpt), int(segments), None, 0)
        workspace = _scratch(workspace, _gated_need(batch, L, dim, dims.dtype, dims.kind, opts.segments, False, False), dev)
        if workspace is not None:
            opts.workspace, opts.workspace_bytes = workspace.data_ptr(), workspace.numel()
        _check(lib.selscan_gated_fwd(_ptr(x), _ptr(g), _ptr(r), _ptr(A), _ptr(z), _ptr(y), _ptr(last_state),
                                     ctypes.byref(dims), ctypes.byref(opts), _stream(dev)))
    return y, last_state


def gated_step(state: torch.Tensor, x: torch.Tensor, g: torch.Tensor, r: Optional[torch.Tensor] = None,
               A: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, *,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the recurrence (selscan_gated_step): updates ``state``
    [batch, dim] fp32 in place and returns y [batch, dim]; ``x``, ``g``, ``r``,
    ``z`` [batch, dim] and ``A`` [dim] as for ``gated_fwd``."""
    if state.dim() != 2:
        raise ValueError("state must be [batch, dim]")
    dev, dt = x.device, x.dtype
    dims = _gated_args(x, g, r, A, z, state.shape)
    _req(state, "state", torch.float32, state.shape, dev)
    with _device(dev):
        if y is None:
            y = torch.empty_like(x)
        else:
            _req(y, "y", dt, state.shape, dev)
        _check(lib.selscan_gated_step(_ptr(state), _ptr(x), _ptr(g), _ptr(r), _ptr(A), _ptr(z), _ptr(y),
                                      ctypes.byref(dims), _stream(dev)))
    return y


def gated_bwd(x: torch.Tensor, g: torch.Tensor, r: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
              z: Optional[torch.Tensor] = None, *, dy: torch.Tensor, h0: Optional[torch.Tensor] = None,
              lengths: Optional[torch.Tensor] = None, dlast_state: Optional[torch.Tensor] = None,
              ckpt: Optional[torch.Tensor] = None, want_dA: bool = True, want_dh0: bool = False, segments: int = 0,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``gated_fwd`` (selscan_gated_bwd) for ``dy`` [batch, L, dim]
    and, when given, ``dlast_state`` (the gradient into last_state).

    Returns a dict with dx, dg and, where there are such inputs, dr, dz (like
    x; 0 behind an entry's length) and dA [dim] fp32, and dh0 [batch, dim] fp32
    when wanted. ``ckpt``: the forward's checkpoints over the same inputs (then
    h0 is not read); without them the states are recomputed. ``workspace``: at
    least ``gated_bwd_workspace_size(...)`` bytes.
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, dim]")
    batch, L, dim = x.shape
    dev = x.device
    dims = _gated_args(x, g, r, A, z, x.shape, dy=dy)
    _req(h0, "h0", torch.float32, (batch, dim), dev)
    _req(dlast_state, "dlast_state", torch.float32, (batch, dim), dev)
    _req(lengths, "lengths", torch.int32, (batch,), dev)
    _req(ckpt, "ckpt", torch.float32, gated_ckpt_shape(batch, L, dim), dev)
    with _device(dev):
        out = {"dx": torch.empty_like(x), "dg": torch.empty_like(x)}
        if r is not None:
            out["dr"] = torch.empty_like(x)
            if want_dA:
                out["dA"] = torch.empty_like(A)
        if z is not None:
            out["dz"] = torch.empty_like(x)
        if want_dh0:
            out["dh0"] = torch.empty((batch, dim), dtype=torch.float32, device=dev)
        opts = GatedBwdOpts(_ptr(h0), _ptr(lengths), _ptr(dlast_state), _ptr(out.get("dh0")), _ptr(ckpt),
                            int(segments), None, 0)
        workspace = _scratch(workspace, _gated_need(batch, L, dim, dims.dtype, dims.kind, opts.segments, True,
                                                    ckpt is not None), dev)
        if workspace is not None:
            opts.workspace, opts.workspace_bytes = workspace.data_ptr(), workspace.numel()
        _check(lib.selscan_gated_bwd(_ptr(x), _ptr(g), _ptr(r), _ptr(A), _ptr(z), _ptr(dy), _ptr(out["dx"]),
                                     _ptr(out["dg"]), _ptr(out.get("dr")), _ptr(out.get("dA")), _ptr(out.get("dz")),
                                     ctypes.byref(dims), ctypes.byref(opts), _stream(dev)))
    return out


NORMS = {"none": 0, "rms": 1, "layer": 2}


def _addnorm_dims(rows, C, dt, res_dt, pre, post, gate, eps, scale, res_scale) -> "AddnormDims":
    if dt not in _DTYPES or res_dt not in _DTYPES:
        raise TypeError(f"unsupported dtypes {dt}, {res_dt}")
    if pre not in NORMS or post not in NORMS:
        raise ValueError(f"pre and post must be one of {sorted(NORMS)}")
    return AddnormDims(rows, C, 0 if gate is None else gate.shape[0], _DTYPES[dt], _DTYPES[res_dt], NORMS[post],
                       NORMS[pre], float(eps), float(scale), float(res_scale))


def _addnorm_opts(C, dev, post_weight, post_bias, pre_weight, pre_bias, gate) -> "AddnormOpts":
    for name, t in (("post_weight", post_weight), ("post_bias", post_bias), ("pre_weight", pre_weight),
                    ("pre_bias", pre_bias)):
        _req(t, name, torch.float32, (C,), dev)
    if gate is not None:
        if gate.dim() != 2 or gate.shape[0] < 1:
            raise ValueError("gate must be [gate_rows, channels], of at least one row")
        _req(gate, "gate", torch.float32, (gate.shape[0], C), dev)
    return AddnormOpts(_ptr(post_weight), _ptr(post_bias), _ptr(pre_weight), _ptr(pre_bias), _ptr(gate), None, 0)


def addnorm(x: torch.Tensor, res: Optional[torch.Tensor] = None, *, pre: str = "rms",
            pre_weight: Optional[torch.Tensor] = None, pre_bias: Optional[torch.Tensor] = None, post: str = "none",
            post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
            gate: Optional[torch.Tensor] = None, scale: float = 1.0, res_scale: float = 1.0, eps: float = 1e-5,
            res_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
            res_out: Optional[torch.Tensor] = None, return_res: bool = True, return_stats: bool = True
            ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The norms around a block with the residual sum (selscan_addnorm). Returns (y, res_out, stats).

    res_out = res_scale res + scale gate post(x) and y = pre(res_out), rounded
    once each; ``post`` and ``pre`` are "none", "rms" or "layer" over the last
    axis, with weights and biases [channels] fp32. ``x`` [..., channels]
    float32 or bfloat16; ``res`` (None: zeros) the same shape, of x's type or
    float32 (``res_dtype`` where there is no res); ``gate`` [gate_rows,
    channels] fp32, each row of it for rows / gate_rows rows of x in turn (None:
    1). ``res_out`` may be ``res`` itself; with ``return_res=False`` it is not
    written. ``stats`` [rows, 4] fp32 is what ``addnorm_bwd`` needs (None with
    ``return_stats=False``). With pre "none" y is None.
    """
    if x.dim() < 1:
        raise ValueError("x must be [..., channels]")
    shape, C, dev, dt = x.shape, x.shape[-1], x.device, x.dtype
    rows = 1
    for n in shape[:-1]:
        rows *= n
    rt = res.dtype if res is not None else res_out.dtype if res_out is not None else res_dtype or dt
    opts = _addnorm_opts(C, dev, post_weight, post_bias, pre_weight, pre_bias, gate)
    dims = _addnorm_dims(rows, C, dt, rt, pre, post, gate, eps, scale, res_scale)
    _req(x, "x", dt, None, dev)
    _req(res, "res", rt, shape, dev)
    with _device(dev):
        if y is not None:
            _req(y, "y", dt, shape, dev)
        elif pre != "none":
            y = torch.empty_like(x)
        if res_out is not None:
            _req(res_out, "res_out", rt, shape, dev)
        elif return_res:
            res_out = torch.empty_like(x if res is None else res, dtype=rt)
        stats = torch.empty((rows, 4), dtype=torch.float32, device=dev) if return_stats else None
        _check(lib.selscan_addnorm(_ptr(x), _ptr(res), _ptr(res_out), _ptr(y), _ptr(stats), ctypes.byref(dims),
                                   ctypes.byref(opts), _stream(dev)))
    return y, res_out, stats


@functools.lru_cache(maxsize=256)
def _addnorm_need(rows: int, C: int, gate_rows: int, dt: int, rt: int, post: int, pre: int, wanted: int) -> int:
    """Bytes of workspace of addnorm_bwd; ``wanted``: a bit for each field of AddnormGrads."""
    dims, n = AddnormDims(rows, C, gate_rows, dt, rt, post, pre, 0.0, 1.0, 1.0), ctypes.c_uint64(0)
    grads = AddnormGrads(*(16 if wanted >> i & 1 else None for i in range(5)))
    _check(lib.selscan_addnorm_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(AddnormOpts(gate=16 if gate_rows else None)),
                                                  ctypes.byref(grads), ctypes.byref(n)))
    return int(n.value)


def addnorm_bwd(x: Optional[torch.Tensor], res_out: Optional[torch.Tensor], *, dy: Optional[torch.Tensor],
                dres_out: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor], pre: str = "rms",
                pre_weight: Optional[torch.Tensor] = None, pre_bias: Optional[torch.Tensor] = None,
                post: str = "none", post_weight: Optional[torch.Tensor] = None,
                post_bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                res_scale: float = 1.0, want_dx: bool = True, want_dres: bool = True, want_dparams: bool = True,
                dres: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                dtype: Optional[torch.dtype] = None, res_dtype: Optional[torch.dtype] = None) -> dict:
    """Gradients of ``addnorm`` (selscan_addnorm_bwd) for ``dy`` (None with pre
    "none") and ``dres_out`` (the gradient into res_out; None: zeros), from the
    ``res_out`` and ``stats`` that it returned.

    Returns a dict with dx, dres (one of them at least; ``dres`` may be
    ``dres_out`` itself) and, with ``want_dparams``, dpost_weight, dpost_bias,
    dpre_weight, dpre_bias [channels] and dgate (like gate), all fp32, of the
    parameters that are given. ``x`` may be None where there is neither a post
    norm nor a gate whose gradient is wanted; with pre "none" ``res_out`` and
    ``dy`` must be None. ``dtype`` is x's type, for dx where neither x nor dy is
    given to say it (None: dres_out's, so a bfloat16 block on a float32 stream
    has to name its own); ``res_dtype`` the residual stream's, for dres where no
    tensor of it is given (None: x's).
    """
    like = next((t for t in (dy, x, res_out, dres_out) if t is not None), None)
    if like is None or like.dim() < 1:
        raise ValueError("dy, x, res_out or dres_out must be given, as [..., channels]")
    shape, C, dev = like.shape, like.shape[-1], like.device
    # (a tensor of another type than the one that is named is turned down below)
    dt = dtype or (dy.dtype if dy is not None else x.dtype if x is not None else like.dtype)
    rt = res_dtype or next((t.dtype for t in (res_out, dres_out, dres) if t is not None), dt)
    rows = 1
    for n in shape[:-1]:
        rows *= n
    opts = _addnorm_opts(C, dev, post_weight, post_bias, pre_weight, pre_bias, gate)
    dims = _addnorm_dims(rows, C, dt, rt, pre, post, gate, 0.0, scale, res_scale)
    for t, name, tt in ((x, "x", dt), (dy, "dy", dt), (res_out, "res_out", rt), (dres_out, "dres_out", rt)):
        _req(t, name, tt, shape, dev)
    _req(stats, "stats", torch.float32, (rows, 4), dev)
    params = dict(post_weight=post_weight, post_bias=post_bias, pre_weight=pre_weight, pre_bias=pre_bias, gate=gate)
    with _device(dev):
        out = {}
        if want_dx:
            out["dx"] = torch.empty(shape, dtype=dt, device=dev)
        if want_dres:
            out["dres"] = torch.empty(shape, dtype=rt, device=dev) if dres is None else dres
            _req(out["dres"], "dres", rt, shape, dev)
        if want_dparams:
            out.update({"d" + n: torch.empty_like(p) for n, p in params.items() if p is not None})
        names = ("dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias", "dgate")
        grads = AddnormGrads(*(_ptr(out.get(n)) for n in names))
        need = _addnorm_need(rows, C, dims.gate_rows, dims.dtype, dims.res_dtype, dims.post, dims.pre,
                             sum(1 << i for i, n in enumerate(names) if n in out))
        workspace = _scratch(workspace, need, dev)
        if workspace is not None:
            opts.workspace, opts.workspace_bytes = workspace.data_ptr(), workspace.numel()
        _check(lib.selscan_addnorm_bwd(_ptr(x), _ptr(res_out), _ptr(stats), _ptr(dy), _ptr(dres_out),
                                       _ptr(out.get("dx")), _ptr(out.get("dres")), ctypes.byref(grads),
                                       ctypes.byref(dims), ctypes.byref(opts), _stream(dev)))
    return out


ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}


def rotary_frequencies(rot: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original: int = 0, fast: float = 32.0, slow: float = 1.0,
                       device: Optional[torch.device] = None) -> torch.Tensor:
    """The ``inv_freq`` [rot / 2] fp32 of ``rotary``: base^(-2 i / rot), for a
    context ``factor`` times as long as the one of training where wanted.

    ``scaling``: "none"; "linear", every frequency divided by ``factor``;
    "base", the base multiplied by factor^(rot / (rot - 2)), which leaves the
    fastest frequency and divides the slowest by ``factor``; "parts", those
    that turn more than ``fast`` times over ``original`` tokens left, those
    that turn less than ``slow`` times divided by ``factor``, and linear in the
    index between these two, each rounded away from the other to a whole index
    from 0 to rot - 1 (the magnitude is ``rotary``'s ``scale``).
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and positive")
    if not (base > 1 and factor > 0):
        raise ValueError("base must be above 1 and factor above 0")
    i = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    if scaling == "base":
        if rot < 4:
            raise ValueError('scaling "base" needs two frequencies')
        base = base * factor ** (rot / (rot - 2))
    freq = float(base) ** -i
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        if original <= 0 or not fast > slow > 0:
            raise ValueError('scaling "parts" needs original > 0 and fast > slow > 0')
        # the index whose frequency turns n times over the original context
        where = [rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (fast, slow)]
        hi = min(math.ceil(where[1]), rot - 1)
        lo = min(max(math.floor(where[0]), 0), hi - 1)  # (hi below 1: all are divided)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / (hi - lo)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
    elif scaling not in ("none", "base"):
        raise ValueError('scaling must be "none", "linear", "base" or "parts"')
    return freq.float().to(device) if device is not None else freq.float()


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: torch.Tensor, *,
           positions: Optional[torch.Tensor] = None, offset: int = 0, layout: str = "half",
           scale: Optional[float] = None, inverse: bool = False, q_out: Optional[torch.Tensor] = None,
           k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions (selscan_rotary). Returns (q_out, k_out).

    ``q`` [batch, L, heads, width], ``k`` [batch, L, kv_heads, width] or None
    (float32 or bfloat16): the first 2 len(inv_freq) values of each head are
    turned by (offset + position) inv_freq, in pairs (i, i + half) or (2 i, 2 i
    + 1) for ``layout`` "half" or "interleaved", and multiplied by ``scale``
    (None: 1). ``positions`` [batch, L] int32 (None: 0, 1, ... along L);
    ``inv_freq`` fp32 (``rotary_frequencies``). ``inverse`` turns back: the
    gradients of q and k are their outputs' gradients turned back. ``q_out``
    and ``k_out`` may be q and k themselves.
    """
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be [batch, L, heads, width]")
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if layout not in ROTARY_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROTARY_LAYOUTS)}")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    if scale is not None and ctypes.c_float(scale).value == 0:
        raise ValueError("scale must not be 0 in fp32 (None: 1)")
    batch, L, H, W = q.shape
    dev, dt = q.device, q.dtype
    Hk = 0 if k is None else k.shape[2]
    _req(q, "q", dt, None, dev)
    _req(k, "k", dt, (batch, L, Hk, W), dev)
    _req(inv_freq, "inv_freq", torch.float32, None, dev)
    _req(positions, "positions", torch.int32, (batch, L), dev)
    dims = RotaryDims(batch, L, H, Hk, W, 2 * inv_freq.shape[0], int(offset), _DTYPES[dt], ROTARY_LAYOUTS[layout],
                      int(inverse), 0.0 if scale is None else float(scale))
    if k is None and k_out is not None:
        raise ValueError("k_out belongs to k")
    with _device(dev):
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            _req(q_out, "q_out", dt, q.shape, dev)
        if k is not None:
            if k_out is None:
                k_out = torch.empty_like(k)
            else:
                _req(k_out, "k_out", dt, k.shape, dev)
        _check(lib.selscan_rotary(_ptr(q), _ptr(k), _ptr(inv_freq), _ptr(positions), _ptr(q_out), _ptr(k_out),
                                  ctypes.byref(dims), _stream(dev)))
    return q_out, k_out


CONV_WIDTH = 4


def conv1d(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
           x_prev: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
           x_last: Optional[torch.Tensor] = None,
           return_x_last: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal depthwise conv1d of width 4 + SiLU (selscan_conv1d). Returns (out, x_last).

    ``x`` [batch, dim, L] (float32 or bfloat16); ``w`` [dim, 4] fp32; ``bias``
    [dim] fp32; ``x_prev`` [batch, dim, 3] fp32, the inputs before token 0
    (None: zeros). ``x_last`` [batch, dim, 3] fp32 receives the last three
    inputs (it may be ``x_prev`` itself).
    """
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    batch, dim, L = x.shape
    dev = x.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    _req(x, "x", x.dtype, (batch, dim, L), dev)
    _req(w, "w", torch.float32, (dim, CONV_WIDTH), dev)
    _req(bias, "bias", torch.float32, (dim,), dev)
    _req(x_prev, "x_prev", torch.float32, (batch, dim, CONV_WIDTH - 1), dev)
    if out is None:
        out = torch.empty_like(x)
    _req(out, "out", x.dtype, (batch, dim, L), dev)
    if x_last is None and return_x_last:
        x_last = torch.empty((batch, dim, CONV_WIDTH - 1), dtype=torch.float32, device=dev)
    _req(x_last, "x_last", torch.float32, (batch, dim, CONV_WIDTH - 1), dev)
    dims = Dims(batch, L, dim, 0, _DTYPES[x.dtype])
    _check(lib.selscan_conv1d(_ptr(x), _ptr(w), _ptr(bias), _ptr(x_prev), _ptr(out), _ptr(x_last),
                              ctypes.byref(dims), _stream(dev)))
    return out, x_last


def conv1d_bwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
               x_prev: Optional[torch.Tensor] = None, *, dout: torch.Tensor,
               want_dbias: bool = True, want_dx_prev: bool = True) -> dict:
    """Gradients of ``conv1d`` (selscan_conv1d_bwd) for ``dout``: a dict with dx
    (like x), dw [dim, 4] fp32, and dbias [dim], dx_prev [batch, dim, 3] fp32
    when wanted."""
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    batch, dim, L = x.shape
    dev = x.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    for t, name, dt, shape in ((x, "x", x.dtype, (batch, dim, L)), (dout, "dout", x.dtype, (batch, dim, L)),
                               (w, "w", torch.float32, (dim, CONV_WIDTH)), (bias, "bias", torch.float32, (dim,)),
                               (x_prev, "x_prev", torch.float32, (batch, dim, CONV_WIDTH - 1))):
        _req(t, name, dt, shape, dev)
    out = {"dx": torch.empty_like(x), "dw": torch.empty((dim, CONV_WIDTH), dtype=torch.float32, device=dev)}
    if want_dbias:
        out["dbias"] = torch.empty((dim,), dtype=torch.float32, device=dev)
    if want_dx_prev:
        out["dx_prev"] = torch.empty((batch, dim, CONV_WIDTH - 1), dtype=torch.float32, device=dev)
    dims = Dims(batch, L, dim, 0, _DTYPES[x.dtype])
    _check(lib.selscan_conv1d_bwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(x_prev), _ptr(dout), _ptr(out["dx"]),
                                  _ptr(out["dw"]), _ptr(out.get("dbias")), _ptr(out.get("dx_prev")),
                                  ctypes.byref(dims), _stream(dev)))
    return out


def conv1d_step(conv_state: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                bias: Optional[torch.Tensor] = None, *,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step of the convolution (selscan_conv1d_step): updates
    ``conv_state`` [batch, dim, 3] fp32 in place and returns out [batch, dim]."""
    if conv_state.dim() != 3:
        raise ValueError("conv_state must be [batch, dim, 3]")
    batch, dim, _ = conv_state.shape
    dev = conv_state.device
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    _req(conv_state, "conv_state", torch.float32, (batch, dim, CONV_WIDTH - 1), dev)
    _req(x, "x", x.dtype, (batch, dim), dev)
    _req(w, "w", torch.float32, (dim, CONV_WIDTH), dev)
    _req(bias, "bias", torch.float32, (dim,), dev)
    if out is None:
        out = torch.empty_like(x)
    _req(out, "out", x.dtype, (batch, dim), dev)
    dims = Dims(batch, 1, dim, 0, _DTYPES[x.dtype])
    _check(lib.selscan_conv1d_step(_ptr(conv_state), _ptr(x), _ptr(w), _ptr(bias), _ptr(out),
                                   ctypes.byref(dims), _stream(dev)))
    return out
