"""Selective state-space scan (the S6 core of Mamba) on MI355X (gfx950).

Thin Python binding over the C ABI in ``include/ssm.h`` (library
``libssm.so``, built in-tree by ``selective_state_space_44_amd._build``).
This module only checks and marshals arguments: tensors are PyTorch device
tensors (PyTorch provides device memory and the current stream); every step
of the computation runs in the HIP kernels.  There is no fallback path: if
the library is missing or a request has no kernel, calls raise.

Entry points: ``scan_fwd`` (the scan; A per channel and the Euler rule as
options; d_state 16, 32, 64, 128), ``scan_fwd_fused`` (with the causal
conv1d + softplus prologue), ``scan_bwd`` and the autograd wrapper
``SelectiveScan`` (all input gradients), ``decode_step`` (one recurrent step
on a resident state), ``ssd_scan`` (step and decay shared per head of 64
channels, on the matrix cores) and its backward ``ssd_bwd``; ``linear_attn``,
``linear_attn_bwd``, ``LinearAttention`` and ``linear_attn_step`` (linear
attention with one decay per head, over prompts, packed sequences and single
tokens), and ``qk_norm_rotate``, ``qk_norm_rotate_bwd``, ``QkNormRotate`` (the
head norm with rotation in front of it); ``gated_delta``, ``gated_delta_bwd``,
``GatedDelta`` and ``gated_delta_step`` (the gated delta rule, likewise), and
``layer_norm``, ``layer_norm_bwd``, ``LayerNorm``.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

import torch
from torch.autograd.function import once_differentiable

__all__ = ["scan_fwd", "scan_fwd_noalloc", "scan_fwd_fused", "scan_bwd", "SelectiveScan", "decode_step", "ssd_scan",
           "ssd_bwd", "linear_attn", "linear_attn_bwd", "LinearAttention", "linear_attn_step",
           "qk_norm_rotate", "qk_norm_rotate_bwd", "QkNormRotate", "gated_delta",
           "gated_delta_bwd", "GatedDelta", "gated_delta_step", "layer_norm", "layer_norm_bwd",
           "LayerNorm",
           "scan_plan", "scan_workspace_bytes", "scan_bwd_workspace_bytes", "load_library",
           "LIB_PATH", "SsmError"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssm.so")

SSM_DTYPE_F32 = 0
SSM_DTYPE_BF16 = 1
SSM_DISC_ZOH = 0
SSM_DISC_EULER = 1
SSM_OK = 0
SSM_ERR_INVALID_ARG = 1
SSM_ERR_UNSUPPORTED = 2
SSM_ERR_WORKSPACE = 3
SSM_ERR_HIP = 4
SSM_NOALLOC_SCRATCH_BYTES = 64 << 20

# Every symbol include/ssm.h declares, with its ctypes signature.
_i64, _vp, _int, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_f32 = ctypes.c_float
SIGNATURES = {
    "ssm_abi_version": (_int, []),
    "ssm_status_str": (ctypes.c_char_p, [_int]),
    "ssm_scan_plan": (_int, [_i64, _i64, _i64, _i64, _int, ctypes.POINTER(_int),
                             ctypes.POINTER(_int), ctypes.POINTER(_int)]),
    "ssm_scan_workspace_bytes": (_i64, [_i64, _i64, _i64, _i64, _int, _int]),
    "ssm_scan_fwd": (_int, [_i64, _i64, _i64, _i64, _int] + [_vp] * 10 + [_vp, _sz, _vp]),
    "ssm_scan_fwd_planned": (_int, [_i64, _i64, _i64, _i64, _int] + [_vp] * 10
                             + [_vp, _sz, _int, _int, _vp]),
    "ssm_scan_fwd_phase": (_int, [_i64, _i64, _i64, _i64, _int] + [_vp] * 10
                           + [_vp, _sz, _int, _int, _int, _vp]),
    "ssm_scan_fwd_noalloc": (_int, [_i64, _i64, _i64, _i64, _int] + [_vp] * 10
                             + [_int, _int, _vp]),
    "ssm_scan_fwd_ex": (_int, [_i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _int, _int]
                        + [_vp] * 7 + [_vp, _sz, _int, _int, _vp]),
    "ssm_scan_fwd_fused": (_int, [_i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _int, _int, _vp,
                                  _vp] + [_vp] * 8 + [_vp, _sz, _int, _int, _vp]),
    "ssm_decode_step": (_int, [_i64, _i64, _i64, _int] + [_vp] * 9 + [_vp]),
    "ssm_decode_step_ex": (_int, [_i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _int, _int]
                           + [_vp] * 6),
    "ssm_scan_bwd_workspace_bytes": (_i64, [_i64, _i64, _i64, _i64, _int]),
    "ssm_scan_bwd": (_int, [_i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _int, _int]
                     + [_vp] * 15 + [_vp, _sz, _vp]),
    "ssm_ssd_fwd": (_int, [_i64, _i64, _i64, _i64, _i64, _int, _int] + [_vp] * 10
                    + [_vp, _sz, _vp]),
    "ssm_ssd_fwd_workspace_bytes": (_i64, [_i64, _i64, _i64, _i64, _i64, _int]),
    "ssm_ssd_fwd_planned": (_int, [_i64, _i64, _i64, _i64, _i64, _int, _int] + [_vp] * 10
                            + [_int, _vp, _sz, _vp]),
    "ssm_ssd_bwd_workspace_bytes": (_i64, [_i64, _i64, _i64, _i64, _i64, _int]),
    "ssm_ssd_bwd": (_int, [_i64, _i64, _i64, _i64, _i64, _int, _int] + [_vp] * 18
                    + [_vp, _sz, _vp]),
    "ssm_linattn_fwd_workspace_bytes": (_i64, [_i64, _i64, _int] + [_i64] * 4 + [_int, _int]),
    "ssm_linattn_fwd": (_int, [_i64, _i64, _vp] + [_i64] * 4 + [_int] + [_vp, _i64] * 3
                        + [_vp, _f32, _vp, _vp, _vp, _int, _vp, _sz, _vp]),
    "ssm_linattn_bwd_workspace_bytes": (_i64, [_i64, _i64, _int] + [_i64] * 4
                                        + [_int, _int, _int]),
    "ssm_linattn_bwd": (_int, [_i64, _i64, _vp] + [_i64] * 4 + [_int] + [_vp, _i64] * 3
                        + [_vp, _f32, _vp, _vp, _i64] + [_vp] * 6 + [_int, _vp, _sz, _vp]),
    "ssm_linattn_step": (_int, [_i64, _i64, _vp] + [_i64] * 4 + [_int, _vp] + [_vp, _i64] * 3
                         + [_vp, _f32, _vp, _vp]),
    "ssm_qk_norm_rotate_fwd": (_int, [_i64] * 6 + [_int, _int] + [_vp, _i64] * 2
                               + [_vp, _vp, _i64, _vp, _vp, _vp, _f32, _vp, _vp, _vp]),
    "ssm_qk_norm_rotate_bwd_workspace_bytes": (_i64, [_i64] * 4),
    "ssm_qk_norm_rotate_bwd": (_int, [_i64] * 6 + [_int, _int] + [_vp, _i64] * 2
                               + [_vp, _vp, _i64, _vp, _vp, _vp, _f32] + [_vp, _i64] * 2
                               + [_vp] * 5 + [_sz, _vp]),
    "ssm_delta_fwd_workspace_bytes": (_i64, [_i64, _i64, _int] + [_i64] * 4 + [_int]),
    "ssm_delta_fwd": (_int, [_i64, _i64, _vp] + [_i64] * 4 + [_int] + [_vp, _i64] * 3
                      + [_vp, _vp, _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "ssm_delta_bwd_workspace_bytes": (_i64, [_i64, _i64, _int] + [_i64] * 4 + [_int]),
    "ssm_delta_bwd": (_int, [_i64, _i64, _vp] + [_i64] * 4 + [_int] + [_vp, _i64] * 3
                      + [_vp, _vp, _f32, _vp, _vp, _i64] + [_vp] * 8 + [_sz, _vp]),
    "ssm_delta_step": (_int, [_i64, _i64, _vp] + [_i64] * 4 + [_int, _vp] + [_vp, _i64] * 3
                       + [_vp, _vp, _f32, _vp, _vp]),
    "ssm_layer_norm_fwd": (_int, [_i64, _i64, _int, _vp, _i64, _vp, _vp, _f32, _vp, _vp]),
    "ssm_layer_norm_bwd_workspace_bytes": (_i64, [_i64, _i64, _int]),
    "ssm_layer_norm_bwd": (_int, [_i64, _i64, _int, _vp, _i64, _vp, _f32, _vp, _i64] + [_vp] * 4
                           + [_sz, _vp]),
}

_lock = threading.Lock()
_lib = None
_calls = None   # the native calls' module
_entry = {}     # addresses of the library's entry points, which they take


class SsmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


def load_library(path: str = LIB_PATH):
    """Load libssm.so (raises OSError if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise OSError(f"{path} is missing: build it with "
                              "`python -m selective_state_space_44_amd._build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
                _entry[name] = ctypes.cast(fn, ctypes.c_void_p).value
            _lib = lib
    return _lib


def status_str(status: int) -> str:
    return load_library().ssm_status_str(int(status)).decode()


def _check(status: int, what: str):
    if status != SSM_OK:
        raise SsmError(status, what)


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return SSM_DTYPE_F32
    if dtype == torch.bfloat16:
        return SSM_DTYPE_BF16
    raise ValueError(f"unsupported I/O dtype {dtype} (float32 or bfloat16)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, name, shape, dtype, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _written(*tensors):
    """Tells autograd that a call has written to tensors of the caller's: one that
    is kept for a backward pass then raises there."""
    for t in tensors:
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def scan_plan(batch: int, seqlen: int, dim: int, dstate: int = 16,
              dtype: torch.dtype = torch.bfloat16, with_phase: bool = False):
    """(waves_per_group, nchunks) that ``scan_fwd`` uses for these sizes; with
    ``with_phase`` also the phase value of its schedule (3: two-launch, 7:
    three-pass, as ``scan_fwd``'s ``phase`` takes them)."""
    g, k, ph = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(load_library().ssm_scan_plan(batch, seqlen, dim, dstate, _io_code(dtype),
                                        ctypes.byref(g), ctypes.byref(k), ctypes.byref(ph)),
           "ssm_scan_plan")
    return (g.value, k.value, ph.value) if with_phase else (g.value, k.value)


def scan_workspace_bytes(batch: int, seqlen: int, dim: int, dstate: int = 16,
                         dtype: torch.dtype = torch.bfloat16, nchunks: int = 0) -> int:
    n = load_library().ssm_scan_workspace_bytes(batch, seqlen, dim, dstate, _io_code(dtype),
                                                nchunks)
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def scan_fwd(x, delta, A, B, C, D=None, z=None, h0=None, return_last_state=False,
             waves_per_group: int = 0, nchunks: int = 0, out=None, workspace=None,
             phase: int = 0, discretization: str = "zoh"):
    """Selective scan.  x, delta, z: [batch, L, dim]; B, C: [batch, L, dstate]
    (all float32 or all bfloat16); A [dim, dstate], D [dim], h0
    [batch, dim, dstate] float32.  Returns y (and the final state when
    ``return_last_state``).  ``waves_per_group``/``nchunks`` override the
    automatic plan (0 = automatic).  ``phase`` 0 runs the whole scan in the
    schedule the plan prefers (``ssm_scan_fwd_planned``); 1, 2 or 3 enqueue
    the first, the second or both launches of the two-launch schedule, 5, 6
    or 7 those of the three-pass schedule (``ssm_scan_fwd_phase``); the
    phases of one scan must get the same ``workspace`` and ``out``.

    Variants (``ssm_scan_fwd_ex``): ``A`` of shape [dim] holds one value per
    channel shared by its states (then ``B``/``C`` fix dstate);
    ``discretization="euler"`` uses Bbar = delta*B instead of the zero-order
    hold.  Both run as one call (``phase`` must be 0), in the plan's schedule."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, seqlen, dim] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    batch, seqlen, dim = x.shape
    if discretization not in ("zoh", "euler"):
        raise ValueError("discretization must be 'zoh' or 'euler'")
    if not isinstance(A, torch.Tensor) or A.dim() not in (1, 2):
        raise ValueError("A must be a [dim, dstate] or [dim] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be a [batch, seqlen, dstate] tensor")
    per_channel = A.dim() == 1
    dstate = B.shape[2] if per_channel else A.shape[1]
    variant = per_channel or discretization != "zoh"
    if variant and phase != 0:
        raise ValueError("the A-per-channel and Euler variants run as one call (phase 0)")
    if phase not in (0, 1, 2, 3, 5, 6, 7):
        raise ValueError("phase must be 0 (the plan's schedule), 1, 2 or 3 (two-launch "
                         "schedule) or 5, 6 or 7 (three-pass schedule)")
    io = x.dtype
    code = _io_code(io)
    _require(x, "x", (batch, seqlen, dim), io, device)
    _require(delta, "delta", (batch, seqlen, dim), io, device)
    _require(A, "A", (dim,) if per_channel else (dim, dstate), torch.float32, device)
    _require(B, "B", (batch, seqlen, dstate), io, device)
    _require(C, "C", (batch, seqlen, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, seqlen, dim), io, device)
    _require(h0, "h0", (batch, dim, dstate), torch.float32, device)
    if delta is None or B is None or C is None:
        raise ValueError("delta, B and C are required")
    y = out if out is not None else torch.empty_like(x)
    _require(y, "out", (batch, seqlen, dim), io, device)
    h_last = (torch.empty((batch, dim, dstate), dtype=torch.float32, device=device)
              if return_last_state else None)
    lib = load_library()
    nbytes = lib.ssm_scan_workspace_bytes(batch, seqlen, dim, dstate, code, nchunks)
    if nbytes < 0:
        raise ValueError("invalid sizes")
    if nbytes > 0 and (workspace is None or workspace.numel() < nbytes):
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if variant:
        st = lib.ssm_scan_fwd_ex(batch, seqlen, dim, dstate, code, _ptr(x), _ptr(delta),
                                 _ptr(A), int(per_channel),
                                 SSM_DISC_EULER if discretization == "euler" else SSM_DISC_ZOH,
                                 _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y),
                                 _ptr(h_last), _ptr(workspace), ws_bytes, int(waves_per_group),
                                 int(nchunks), _stream(device))
        _check(st, "ssm_scan_fwd_ex")
        return (y, h_last) if return_last_state else y
    if phase == 0:
        st = lib.ssm_scan_fwd_planned(batch, seqlen, dim, dstate, code, _ptr(x), _ptr(delta),
                                      _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0),
                                      _ptr(y), _ptr(h_last), _ptr(workspace), ws_bytes,
                                      int(waves_per_group), int(nchunks), _stream(device))
        _check(st, "ssm_scan_fwd_planned")
    else:
        st = lib.ssm_scan_fwd_phase(batch, seqlen, dim, dstate, code, _ptr(x), _ptr(delta),
                                    _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0),
                                    _ptr(y), _ptr(h_last), _ptr(workspace), ws_bytes,
                                    int(waves_per_group), int(nchunks), int(phase),
                                    _stream(device))
        _check(st, "ssm_scan_fwd_phase")
    return (y, h_last) if return_last_state else y


def scan_fwd_noalloc(x, delta, A, B, C, D=None, z=None, h0=None, *, out,
                     h_last=None, waves_per_group: int = 0, nchunks: int = 0):
    """``ssm_scan_fwd_noalloc``: the scan of ``scan_fwd`` (per-state A, zero-
    order hold) with its chunk-carry workspace in the library's device scratch
    array, so that the call allocates nothing: the caller passes the output
    ``out`` [batch, L, dim] and, optionally, ``h_last`` [batch, dim, dstate]
    float32.  Raises SsmError(SSM_ERR_WORKSPACE) when the plan's workspace
    exceeds SSM_NOALLOC_SCRATCH_BYTES.  Calls that overlap on one GPU race on
    the scratch array."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, seqlen, dim] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    batch, seqlen, dim = x.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [dim, dstate] tensor")
    dstate = A.shape[1]
    io = x.dtype
    code = _io_code(io)
    _require(x, "x", (batch, seqlen, dim), io, device)
    _require(delta, "delta", (batch, seqlen, dim), io, device)
    _require(A, "A", (dim, dstate), torch.float32, device)
    _require(B, "B", (batch, seqlen, dstate), io, device)
    _require(C, "C", (batch, seqlen, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, seqlen, dim), io, device)
    _require(h0, "h0", (batch, dim, dstate), torch.float32, device)
    _require(out, "out", (batch, seqlen, dim), io, device)
    _require(h_last, "h_last", (batch, dim, dstate), torch.float32, device)
    if delta is None or B is None or C is None or out is None:
        raise ValueError("delta, B, C and out are required")
    st = load_library().ssm_scan_fwd_noalloc(
        batch, seqlen, dim, dstate, code, _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C),
        _ptr(D), _ptr(z), _ptr(h0), _ptr(out), _ptr(h_last), int(waves_per_group),
        int(nchunks), _stream(device))
    _check(st, "ssm_scan_fwd_noalloc")
    return out


def ssd_scan(x, dt, A, B, C, D=None, z=None, h0=None, return_last_state=False,
             discretization: str = "zoh", out=None, nsplit: int = 0, workspace=None):
    """Scan with the step and decay rate shared by each head
    (``ssm_ssd_fwd_planned``).  x, z: [batch, L, nheads * headdim]; dt:
    [batch, L, nheads]; B, C: [batch, L, dstate] (all bfloat16); A [nheads],
    D [nheads * headdim], h0 [batch, nheads * headdim, dstate] float32.
    headdim = x.shape[2] // dt.shape[2].  ``nsplit`` sequence segments (0 =
    automatic, 1 = none).  Returns y (and the final state when
    ``return_last_state``)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, seqlen, dim] tensor")
    if not isinstance(dt, torch.Tensor) or dt.dim() != 3:
        raise ValueError("dt must be a [batch, seqlen, nheads] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be a [batch, seqlen, dstate] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    if discretization not in ("zoh", "euler"):
        raise ValueError("discretization must be 'zoh' or 'euler'")
    batch, seqlen, dim = x.shape
    nheads = dt.shape[2]
    if nheads == 0 or dim % nheads:
        raise ValueError("x's channels must split evenly into dt's heads")
    headdim = dim // nheads
    dstate = B.shape[2]
    io = x.dtype
    code = _io_code(io)
    _require(x, "x", (batch, seqlen, dim), io, device)
    _require(dt, "dt", (batch, seqlen, nheads), io, device)
    _require(A, "A", (nheads,), torch.float32, device)
    _require(B, "B", (batch, seqlen, dstate), io, device)
    _require(C, "C", (batch, seqlen, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, seqlen, dim), io, device)
    _require(h0, "h0", (batch, dim, dstate), torch.float32, device)
    if A is None or C is None:
        raise ValueError("A and C are required")
    y = out if out is not None else torch.empty_like(x)
    _require(y, "out", (batch, seqlen, dim), io, device)
    h_last = (torch.empty((batch, dim, dstate), dtype=torch.float32, device=device)
              if return_last_state else None)
    lib = load_library()
    nbytes = lib.ssm_ssd_fwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, int(nsplit))
    if nbytes < 0:
        raise ValueError("invalid sizes")
    if nbytes > 0 and (workspace is None or workspace.numel() < nbytes):
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssm_ssd_fwd_planned(
        batch, seqlen, nheads, headdim, dstate, code,
        SSM_DISC_EULER if discretization == "euler" else SSM_DISC_ZOH, _ptr(x), _ptr(dt),
        _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last),
        int(nsplit), _ptr(workspace), ws_bytes, _stream(device))
    _check(st, "ssm_ssd_fwd_planned")
    return (y, h_last) if return_last_state else y


def ssd_bwd(x, dt, A, B, C, D=None, z=None, h0=None, *, dy, dh_last=None,
            discretization: str = "zoh", need_dD: bool = True, need_dh0: bool = True,
            workspace=None):
    """Gradients of ``ssd_scan`` for upstream dy (and dh_last).  Returns a dict:
    dx, dz (None without z), ddt, dB, dC in the I/O dtype; dA [nheads], dD
    (None unless need_dD), dh0 (None unless need_dh0) in float32."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, seqlen, dim] tensor")
    if not isinstance(dt, torch.Tensor) or dt.dim() != 3:
        raise ValueError("dt must be a [batch, seqlen, nheads] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be a [batch, seqlen, dstate] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    if discretization not in ("zoh", "euler"):
        raise ValueError("discretization must be 'zoh' or 'euler'")
    batch, seqlen, dim = x.shape
    nheads = dt.shape[2]
    if nheads == 0 or dim % nheads:
        raise ValueError("x's channels must split evenly into dt's heads")
    headdim, dstate = dim // nheads, B.shape[2]
    io = x.dtype
    code = _io_code(io)
    _require(x, "x", (batch, seqlen, dim), io, device)
    _require(dt, "dt", (batch, seqlen, nheads), io, device)
    _require(A, "A", (nheads,), torch.float32, device)
    _require(B, "B", (batch, seqlen, dstate), io, device)
    _require(C, "C", (batch, seqlen, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, seqlen, dim), io, device)
    _require(h0, "h0", (batch, dim, dstate), torch.float32, device)
    _require(dy, "dy", (batch, seqlen, dim), io, device)
    _require(dh_last, "dh_last", (batch, dim, dstate), torch.float32, device)
    if A is None or C is None or dy is None:
        raise ValueError("A, C and dy are required")
    g = {
        "dx": torch.empty_like(x), "ddt": torch.empty_like(dt),
        "dz": torch.empty_like(x) if z is not None else None,
        "dA": torch.empty_like(A), "dB": torch.empty_like(B), "dC": torch.empty_like(C),
        "dD": torch.empty(dim, dtype=torch.float32, device=device) if need_dD else None,
        "dh0": (torch.empty((batch, dim, dstate), dtype=torch.float32, device=device)
                if need_dh0 else None),
    }
    lib = load_library()
    nbytes = lib.ssm_ssd_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, code)
    if nbytes < 0:
        raise ValueError("invalid sizes")
    if nbytes > 0 and (workspace is None or workspace.numel() < nbytes):
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssm_ssd_bwd(batch, seqlen, nheads, headdim, dstate, code,
                         SSM_DISC_EULER if discretization == "euler" else SSM_DISC_ZOH,
                         _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                         _ptr(h0), _ptr(dy), _ptr(dh_last), _ptr(g["dx"]), _ptr(g["ddt"]),
                         _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
                         _ptr(g["dz"]), _ptr(g["dh0"]), _ptr(workspace), ws_bytes,
                         _stream(device))
    _check(st, "ssm_ssd_bwd")
    return g


def scan_fwd_fused(x_raw, conv_w, conv_b, delta_raw, delta_bias, A, B, C, D=None, z=None,
                   h0=None, *, conv_silu: bool, return_last_state=False,
                   waves_per_group: int = 0, nchunks: int = 0, out=None, workspace=None):
    """Selective scan with its prologue fused: x = act(causal depthwise
    conv1d(x_raw) + conv_b), delta = softplus(delta_raw + delta_bias), then the
    scan of ``scan_fwd``.  x_raw, delta_raw: [batch, L, dim] (float32 or
    bfloat16); conv_w [dim, d_conv] float32 (d_conv <= 4, the last tap
    multiplies the current step); conv_b, delta_bias [dim] float32 or None;
    ``conv_silu`` selects SiLU after the convolution (keyword, no default)."""
    if not isinstance(x_raw, torch.Tensor) or x_raw.dim() != 3:
        raise ValueError("x_raw must be a [batch, seqlen, dim] tensor")
    device = x_raw.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    batch, seqlen, dim = x_raw.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [dim, dstate] tensor")
    if not isinstance(conv_w, torch.Tensor) or conv_w.dim() != 2:
        raise ValueError("conv_w must be a [dim, d_conv] tensor")
    dstate = A.shape[1]
    d_conv = conv_w.shape[1]
    io = x_raw.dtype
    code = _io_code(io)
    _require(x_raw, "x_raw", (batch, seqlen, dim), io, device)
    _require(delta_raw, "delta_raw", (batch, seqlen, dim), io, device)
    _require(conv_w, "conv_w", (dim, d_conv), torch.float32, device)
    _require(conv_b, "conv_b", (dim,), torch.float32, device)
    _require(delta_bias, "delta_bias", (dim,), torch.float32, device)
    _require(A, "A", (dim, dstate), torch.float32, device)
    _require(B, "B", (batch, seqlen, dstate), io, device)
    _require(C, "C", (batch, seqlen, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, seqlen, dim), io, device)
    _require(h0, "h0", (batch, dim, dstate), torch.float32, device)
    if delta_raw is None or B is None or C is None:
        raise ValueError("delta_raw, B and C are required")
    y = out if out is not None else torch.empty_like(x_raw)
    _require(y, "out", (batch, seqlen, dim), io, device)
    h_last = (torch.empty((batch, dim, dstate), dtype=torch.float32, device=device)
              if return_last_state else None)
    lib = load_library()
    nbytes = lib.ssm_scan_workspace_bytes(batch, seqlen, dim, dstate, code, nchunks)
    if nbytes < 0:
        raise ValueError("invalid sizes")
    if nbytes > 0 and (workspace is None or workspace.numel() < nbytes):
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssm_scan_fwd_fused(batch, seqlen, dim, dstate, code, _ptr(x_raw), _ptr(conv_w),
                                _ptr(conv_b), int(d_conv), int(bool(conv_silu)),
                                _ptr(delta_raw), _ptr(delta_bias), _ptr(A), _ptr(B), _ptr(C),
                                _ptr(D), _ptr(z), _ptr(h0), _ptr(y), _ptr(h_last),
                                _ptr(workspace), ws_bytes, int(waves_per_group), int(nchunks),
                                _stream(device))
    _check(st, "ssm_scan_fwd_fused")
    return (y, h_last) if return_last_state else y


def decode_step(h, x, delta, A, B, C, D=None, z=None, out=None, discretization: str = "zoh"):
    """One recurrent step.  h: [batch, dim, dstate] float32, updated in place;
    x, delta, z: [batch, dim]; B, C: [batch, dstate] (float32 or bfloat16);
    A [dim, dstate] (or [dim]: one value per channel), D [dim] float32.
    ``discretization="euler"`` uses Bbar = delta*B.  Returns y [batch, dim]."""
    if not isinstance(h, torch.Tensor) or h.dim() != 3:
        raise ValueError("h must be a [batch, dim, dstate] tensor")
    device = h.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    if discretization not in ("zoh", "euler"):
        raise ValueError("discretization must be 'zoh' or 'euler'")
    batch, dim, dstate = h.shape
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a tensor")
    if not isinstance(A, torch.Tensor) or A.dim() not in (1, 2):
        raise ValueError("A must be a [dim, dstate] or [dim] tensor")
    per_channel = A.dim() == 1
    io = x.dtype
    code = _io_code(io)
    _require(h, "h", (batch, dim, dstate), torch.float32, device)
    _require(x, "x", (batch, dim), io, device)
    _require(delta, "delta", (batch, dim), io, device)
    _require(A, "A", (dim,) if per_channel else (dim, dstate), torch.float32, device)
    _require(B, "B", (batch, dstate), io, device)
    _require(C, "C", (batch, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, dim), io, device)
    if delta is None or B is None or C is None:
        raise ValueError("delta, B and C are required")
    y = out if out is not None else torch.empty_like(x)
    _require(y, "out", (batch, dim), io, device)
    lib = load_library()
    if per_channel or discretization != "zoh":
        st = lib.ssm_decode_step_ex(batch, dim, dstate, code, _ptr(h), _ptr(x), _ptr(delta),
                                    _ptr(A), int(per_channel),
                                    SSM_DISC_EULER if discretization == "euler" else SSM_DISC_ZOH,
                                    _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), _stream(device))
        _check(st, "ssm_decode_step_ex")
        _written(h)
        return y
    st = lib.ssm_decode_step(batch, dim, dstate, code, _ptr(h), _ptr(x), _ptr(delta), _ptr(A),
                             _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), _stream(device))
    _check(st, "ssm_decode_step")
    _written(h)
    return y


def scan_bwd_workspace_bytes(batch: int, seqlen: int, dim: int, dstate: int = 16,
                             dtype: torch.dtype = torch.bfloat16) -> int:
    n = load_library().ssm_scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, _io_code(dtype))
    if n < 0:
        raise ValueError("invalid sizes")
    return int(n)


def scan_bwd(x, delta, A, B, C, D=None, z=None, h0=None, *, dy, dh_last=None,
             discretization: str = "zoh", need_dD: bool = True, need_dh0: bool = True,
             workspace=None):
    """Gradients of the scan for upstream dy [batch, L, dim] (and dh_last
    [batch, dim, dstate] float32).  Inputs as ``scan_fwd``.  Returns a dict:
    dx, ddelta, dz (None without z) [batch, L, dim] and dB, dC [batch, L,
    dstate] in the I/O dtype; dA (shape of A), dD [dim] (None unless
    need_dD), dh0 [batch, dim, dstate] (None unless need_dh0) in float32."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [batch, seqlen, dim] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    batch, seqlen, dim = x.shape
    if discretization not in ("zoh", "euler"):
        raise ValueError("discretization must be 'zoh' or 'euler'")
    if not isinstance(A, torch.Tensor) or A.dim() not in (1, 2):
        raise ValueError("A must be a [dim, dstate] or [dim] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be a [batch, seqlen, dstate] tensor")
    per_channel = A.dim() == 1
    dstate = B.shape[2] if per_channel else A.shape[1]
    io = x.dtype
    code = _io_code(io)
    _require(x, "x", (batch, seqlen, dim), io, device)
    _require(delta, "delta", (batch, seqlen, dim), io, device)
    _require(A, "A", (dim,) if per_channel else (dim, dstate), torch.float32, device)
    _require(B, "B", (batch, seqlen, dstate), io, device)
    _require(C, "C", (batch, seqlen, dstate), io, device)
    _require(D, "D", (dim,), torch.float32, device)
    _require(z, "z", (batch, seqlen, dim), io, device)
    _require(h0, "h0", (batch, dim, dstate), torch.float32, device)
    _require(dy, "dy", (batch, seqlen, dim), io, device)
    _require(dh_last, "dh_last", (batch, dim, dstate), torch.float32, device)
    if delta is None or C is None or dy is None:
        raise ValueError("delta, C and dy are required")
    g = {
        "dx": torch.empty_like(x), "ddelta": torch.empty_like(x),
        "dz": torch.empty_like(x) if z is not None else None,
        "dA": torch.empty_like(A), "dB": torch.empty_like(B), "dC": torch.empty_like(C),
        "dD": torch.empty(dim, dtype=torch.float32, device=device) if need_dD else None,
        "dh0": (torch.empty((batch, dim, dstate), dtype=torch.float32, device=device)
                if need_dh0 else None),
    }
    lib = load_library()
    nbytes = lib.ssm_scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, code)
    if nbytes < 0:
        raise ValueError("invalid sizes")
    if nbytes > 0 and (workspace is None or workspace.numel() < nbytes):
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssm_scan_bwd(batch, seqlen, dim, dstate, code, _ptr(x), _ptr(delta), _ptr(A),
                          int(per_channel),
                          SSM_DISC_EULER if discretization == "euler" else SSM_DISC_ZOH,
                          _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(h0), _ptr(dy),
                          _ptr(dh_last), _ptr(g["dx"]), _ptr(g["ddelta"]), _ptr(g["dA"]),
                          _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]), _ptr(g["dz"]),
                          _ptr(g["dh0"]), _ptr(workspace), ws_bytes, _stream(device))
    _check(st, "ssm_scan_bwd")
    return g


def _as_operand(t):
    """A gradient as the kernels take it, contiguous from a 16-byte boundary:
    autograd may hand in a piece of another tensor."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class SelectiveScan(torch.autograd.Function):
    """Autograd wrapper: forward = ``scan_fwd`` (returns y and h_last),
    backward = ``scan_bwd``; both run the HIP kernels only.

    ``y, h_last = SelectiveScan.apply(x, delta, A, B, C, D, z, h0, discretization)``
    (D, z, h0 may be None).  Differentiable once."""

    @staticmethod
    def forward(ctx, x, delta, A, B, C, D, z, h0, discretization="zoh"):
        y, h_last = scan_fwd(x, delta, A, B, C, D, z, h0, return_last_state=True,
                             discretization=discretization)
        ctx.save_for_backward(x, delta, A, B, C, D, z, h0)
        ctx.discretization = discretization
        return y, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        x, delta, A, B, C, D, z, h0 = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        g = scan_bwd(x, delta, A, B, C, D, z, h0, dy=_as_operand(dy),
                     dh_last=None if dh_last is None else _as_operand(dh_last),
                     discretization=ctx.discretization,
                     need_dD=D is not None and ctx.needs_input_grad[5],
                     need_dh0=h0 is not None and ctx.needs_input_grad[7])
        return (g["dx"], g["ddelta"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["dh0"],
                None)


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(device):
    """The current stream's handle (as ``_stream``, without building objects:
    the calls below are made once per token and layer)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _library():
    return _lib or load_library()


def _native():
    """The native calls, which only the functions below need (raises OSError if
    they have not been built, or for another torch)."""
    global _calls
    if _lib is None:
        load_library()
    if _calls is None:
        with _lock:
            try:
                _calls = importlib.import_module("._calls", __name__)
            except ImportError as e:
                raise OSError("the native calls are missing: build them with "
                              "`python -m selective_state_space_44_amd._build`") from e
    return _calls


def _outputs(r, what):
    """A native call's outputs; None when it left the call to the checks here."""
    if r.__class__ is int:
        _check(r, what)
    return r


def _given(t, name, shape, dtype, device):
    """``_require`` for a tensor that is there, quick when it is as it should be."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape \
            and t.get_device() == device.index and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name} is required")
    _require(t, name, shape, dtype, device)
    return t.data_ptr()


def _optional(t, name, shape, dtype, device):
    return None if t is None else _given(t, name, shape, dtype, device)


_WHOLE = torch.contiguous_format


def _new(t, shape):
    """A contiguous tensor of t's type and device: ``empty_like`` takes a
    microsecond less than ``empty``."""
    return torch.empty_like(t, memory_format=_WHOLE) if t.shape == shape else t.new_empty(shape)


def _strided(t, name, shape, dtype, device):
    """Address of a [..., tokens, heads, dim] tensor whose last two dimensions
    are contiguous and whose tokens are evenly spaced (a slice of a fused
    projection, for instance), and the elements between its tokens."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == device.index):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch.Tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr(), _token_stride(t, name, shape)


def _token_stride(t, name, shape):
    heads, dim = shape[-2], shape[-1]
    if t.is_contiguous():
        return heads * dim
    s = t.stride()
    # a dimension of one element may have any stride
    if (s[-1] != 1 and dim > 1) or (s[-2] != dim and heads > 1):
        raise ValueError(f"{name}'s heads must be contiguous")
    if len(shape) == 3 or shape[0] == 1:
        return s[-3] if shape[-3] > 1 else heads * dim
    if shape[1] == 1:
        return s[0]
    if s[0] != shape[1] * s[1]:
        raise ValueError(f"{name}'s tokens must be evenly spaced")
    return s[1]


def _linattn_args(q, k, v, log_decay, h0, cu_seqlens):
    """Checked operands of the whole-sequence calls: (shape of q without its
    channels, sizes for the workspace, arguments up to h0, state shape)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{n} must be a torch.Tensor")
    nd = 4 if cu_seqlens is None else 3
    if q.dim() != nd or k.dim() != nd or v.dim() != nd:
        raise ValueError("q, k and v must be [batch, seqlen, heads, dim] tensors, or [tokens, "
                         "heads, dim] with cu_seqlens")
    device = q.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    *lead, heads, kdim = q.shape
    kv, vdim = k.shape[-2], v.shape[-1]
    if cu_seqlens is None:
        batch, seqlen = lead
        cu = None
    else:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 \
                or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a [sequences + 1] tensor")
        cu = _given(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, device)
        batch, seqlen = cu_seqlens.numel() - 1, lead[0]
        if batch == 0 and seqlen > 0:
            raise ValueError("tokens without a sequence")
    if heads and (kv == 0 or heads % kv):
        raise ValueError("q's heads must split evenly over k's")
    io = q.dtype
    code = _io_code(io)
    state = (batch, heads, vdim, kdim)
    args = (batch, seqlen, cu, heads, kv, kdim, vdim, code,
            q.data_ptr(), _token_stride(q, "q", q.shape),
            *_strided(k, "k", (*lead, kv, kdim), io, device),
            *_strided(v, "v", (*lead, kv, vdim), io, device),
            _given(log_decay, "log_decay", (heads,), torch.float32, device))
    sizes = (batch, seqlen, cu is not None, heads, kv, kdim, vdim, code)
    return (*lead, heads), sizes, args, state, _optional(h0, "h0", state, torch.float32, device)


def _workspace(nbytes, workspace, device):
    if nbytes < 0:
        raise ValueError("unsupported sizes")
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise ValueError("workspace must be a torch.Tensor")
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, expected {device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def linear_attn(q, k, v, log_decay, h0=None, *, scale: float = 1.0, cu_seqlens=None,
                return_last_state=False, nsplit: int = 0, out=None, workspace=None):
    """Linear attention with one decay per head (``ssm_linattn_fwd``):
    S_t = exp(log_decay) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.  q
    [batch, L, heads, kdim], k [batch, L, kv_heads, kdim], v [batch, L,
    kv_heads, vdim] (float32 or bfloat16; tokens may be strided), or without
    the batch dimension and with ``cu_seqlens`` (int32 [sequences + 1] on the
    device, from 0 to the number of tokens; outputs and gradients of tokens that
    no sequence holds are not written) for packed sequences; log_decay [heads], h0 [sequences, heads,
    vdim, kdim] float32.  ``nsplit`` segments per sequence (0 = automatic:
    packed, by the mean length; give it where one is much longer than the
    others).  Returns o [batch, L, heads, vdim] (and the final state when
    ``return_last_state``)."""
    if out is None and workspace is None:
        r = _outputs(_native().linattn_fwd(
            _entry["ssm_linattn_fwd"], _entry["ssm_linattn_fwd_workspace_bytes"], q, k, v,
            log_decay, h0, cu_seqlens, scale, return_last_state, nsplit), "ssm_linattn_fwd")
        if r is not None:
            return r if return_last_state else r[0]
    lead, sizes, args, state, h0_at = _linattn_args(q, k, v, log_decay, h0, cu_seqlens)
    device, io = q.device, q.dtype
    shape = (*lead, v.shape[-1])
    if out is None:
        out = _new(q, shape)
        o_at = out.data_ptr()
    else:
        o_at = _given(out, "out", shape, io, device)
    h_last = torch.empty(state, dtype=torch.float32, device=device) if return_last_state else None
    lib = _library()
    ws, ws_bytes, keep = _workspace(lib.ssm_linattn_fwd_workspace_bytes(*sizes, nsplit), workspace,
                                    device)
    st = lib.ssm_linattn_fwd(*args, scale, h0_at, o_at, _addr(h_last), nsplit, ws, ws_bytes,
                             _raw_stream(device))
    if st:
        _check(st, "ssm_linattn_fwd")
    _written(out)
    return (out, h_last) if return_last_state else out


def linear_attn_bwd(q, k, v, log_decay, h0=None, *, dy, dh_last=None, scale: float = 1.0,
                    cu_seqlens=None, need_dlog_decay: bool = False, need_dh0: bool = True,
                    nsplit: int = 0, workspace=None):
    """Gradients of ``linear_attn`` for upstream dy (and dh_last).  Returns a
    dict: dq, dk, dv in the I/O dtype (dk and dv summed over the query heads
    that share them); dlog_decay [heads] (None unless need_dlog_decay) and dh0
    (None unless need_dh0) in float32."""
    if workspace is None:
        r = _outputs(_native().linattn_bwd(
            _entry["ssm_linattn_bwd"], _entry["ssm_linattn_bwd_workspace_bytes"], q, k, v,
            log_decay, h0, cu_seqlens, scale, dy, dh_last, need_dlog_decay, need_dh0, nsplit),
            "ssm_linattn_bwd")
        if r is not None:
            return dict(zip(("dq", "dk", "dv", "dlog_decay", "dh0"), r))
    lead, sizes, args, state, h0_at = _linattn_args(q, k, v, log_decay, h0, cu_seqlens)
    device, io = q.device, q.dtype
    dy_at = _strided(dy, "dy", (*lead, v.shape[-1]), io, device)
    dh_at = _optional(dh_last, "dh_last", state, torch.float32, device)

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=device)
    g = {"dq": torch.empty_like(q, memory_format=_WHOLE),
         "dk": torch.empty_like(k, memory_format=_WHOLE),
         "dv": torch.empty_like(v, memory_format=_WHOLE),
         "dlog_decay": new(lead[-1], torch.float32) if need_dlog_decay else None,
         "dh0": new(state, torch.float32) if need_dh0 else None}
    lib = _library()
    ws, ws_bytes, keep = _workspace(
        lib.ssm_linattn_bwd_workspace_bytes(*sizes, bool(need_dlog_decay), nsplit), workspace,
        device)
    st = lib.ssm_linattn_bwd(*args, scale, h0_at, *dy_at, dh_at, _addr(g["dq"]), _addr(g["dk"]),
                             _addr(g["dv"]), _addr(g["dlog_decay"]), _addr(g["dh0"]), nsplit, ws,
                             ws_bytes, _raw_stream(device))
    if st:
        _check(st, "ssm_linattn_bwd")
    return g


def linear_attn_step(h, q, k, v, log_decay, *, scale: float = 1.0, slots=None, out=None):
    """One token of ``linear_attn`` per row on resident states
    (``ssm_linattn_step``).  h [nslots, heads, vdim, kdim] float32, updated in
    place; q [batch, heads, kdim], k [batch, kv_heads, kdim], v [batch,
    kv_heads, vdim]; ``slots`` int32 [batch] names each row's state (None: row
    b uses slot b; a row with a slot outside [0, nslots) answers zeros).
    Returns o [batch, heads, vdim]."""
    if out is None:
        r = _outputs(_native().linattn_step(_entry["ssm_linattn_step"], h, q, k, v, log_decay,
                                            scale, slots), "ssm_linattn_step")
        if r is not None:
            return r[0]
    if not isinstance(h, torch.Tensor) or h.dim() != 4:
        raise ValueError("h must be a [nslots, heads, vdim, kdim] tensor")
    device = h.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 3 \
            or k.dim() != 3:
        raise ValueError("q, k and v must be [batch, heads, dim] tensors")
    nslots, heads, vdim, kdim = h.shape
    batch, kv = q.shape[0], k.shape[1]
    if heads and (kv == 0 or heads % kv):
        raise ValueError("q's heads must split evenly over k's")
    if slots is None and nslots < batch:
        raise ValueError(f"h holds {nslots} states for {batch} rows")
    io = q.dtype
    shape = (batch, heads, vdim)
    if out is None:
        out = _new(q, shape)
        o_at = out.data_ptr()
    else:
        o_at = _given(out, "out", shape, io, device)
    st = _library().ssm_linattn_step(
        batch, nslots, _optional(slots, "slots", (batch,), torch.int32, device), heads, kv, kdim,
        vdim, _io_code(io), _given(h, "h", h.shape, torch.float32, device),
        *_strided(q, "q", (batch, heads, kdim), io, device),
        *_strided(k, "k", (batch, kv, kdim), io, device),
        *_strided(v, "v", (batch, kv, vdim), io, device),
        _given(log_decay, "log_decay", (heads,), torch.float32, device), scale, o_at,
        _raw_stream(device))
    if st:
        _check(st, "ssm_linattn_step")
    _written(h, out)
    return out


class LinearAttention(torch.autograd.Function):
    """Autograd wrapper of ``linear_attn``: apply(q, k, v, log_decay, h0,
    scale, cu_seqlens) -> (o, h_last); h0 and cu_seqlens may be None.
    Differentiable once; scale is a number, without a gradient."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, h0=None, scale=1.0, cu_seqlens=None):
        o, h_last = linear_attn(q, k, v, log_decay, h0, scale=scale, cu_seqlens=cu_seqlens,
                                return_last_state=True)
        ctx.save_for_backward(q, k, v, log_decay, h0, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        if any(ctx.needs_input_grad[5:6]):
            raise ValueError("scale has no gradient: detach it, or scale q")
        q, k, v, log_decay, h0, cu_seqlens = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros((*q.shape[:-1], v.shape[-1]), dtype=q.dtype, device=q.device)
        if dh_last is not None:
            dh_last = _as_operand(dh_last)
        g = linear_attn_bwd(q, k, v, log_decay, h0, dy=_as_operand(dy), dh_last=dh_last,
                            scale=ctx.scale, cu_seqlens=cu_seqlens,
                            need_dlog_decay=ctx.needs_input_grad[3],
                            need_dh0=h0 is not None and ctx.needs_input_grad[4])
        return g["dq"], g["dk"], g["dv"], g["dlog_decay"], g["dh0"], None, None


def _rotate_args(q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved):
    """Checked arguments up to eps of the norm-and-rotation calls."""
    if not (isinstance(q, torch.Tensor) and isinstance(k, torch.Tensor)):
        raise ValueError("q and k must be torch.Tensors")
    shape, kshape, device, io = q.shape, k.shape, q.device, q.dtype
    if len(shape) not in (3, 4) or len(kshape) != len(shape):
        raise ValueError("q and k must be [batch, seqlen, heads, dim] or [tokens, heads, dim] "
                         "tensors")
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    dim, hk, seqlen, f32 = shape[-1], kshape[-2], shape[-3], torch.float32
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    npos = half = 0
    cos_at = sin_at = None
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a [positions, rot / 2] tensor")
        table = cos.shape
        npos, half = table
        cos_at = _given(cos, "cos", table, f32, device)
        sin_at = _given(sin, "sin", table, f32, device)
    if half and positions is None and seqlen > npos:
        raise ValueError(f"the rotation table has {npos} positions, the sequence {seqlen}")
    lead = shape[:-2]
    k_at, k_stride = _strided(k, "k", (*lead, hk, dim), io, device)
    return (seqlen if len(shape) == 3 else shape[0] * seqlen, seqlen, shape[-2], hk, dim, 2 * half,
            1 if interleaved else 0, _io_code(io), q.data_ptr(), _token_stride(q, "q", shape),
            k_at, k_stride, cos_at, sin_at, npos, None if positions is None else
            _given(positions, "positions", lead, torch.int64, device),
            None if q_weight is None else _given(q_weight, "q_weight", (dim,), f32, device),
            None if k_weight is None else _given(k_weight, "k_weight", (dim,), f32, device), eps)


def qk_norm_rotate(q, k, cos, sin, positions=None, q_weight=None, k_weight=None, *,
                   eps: float = 1e-6, interleaved: bool = False, out=None):
    """RMS norm of every query and key head and the rotation by the token's
    position in one pass (``ssm_qk_norm_rotate_fwd``).  q [batch, L, heads,
    dim], k [batch, L, kv_heads, dim] (or [tokens, heads, dim]; float32 or
    bfloat16; tokens may be strided); cos, sin [positions, rot / 2] float32
    (None: no rotation); positions int64 [batch, L] (None: 0 .. L - 1);
    q_weight, k_weight [dim] float32 or None.  Pairs are channels (i, i +
    rot / 2), or (2i, 2i + 1) when ``interleaved``.  Returns (q, k);
    ``out`` takes a pair of tensors for them."""
    if out is None:
        r = _outputs(_native().rotate_fwd(_entry["ssm_qk_norm_rotate_fwd"], q, k, cos, sin,
                                          positions, q_weight, k_weight, eps, interleaved),
                     "ssm_qk_norm_rotate_fwd")
        if r is not None:
            return r
    args = _rotate_args(q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved)
    device, io = q.device, q.dtype
    if out is None:
        qo = torch.empty_like(q, memory_format=_WHOLE)
        ko = torch.empty_like(k, memory_format=_WHOLE)
        at = qo.data_ptr(), ko.data_ptr()
    else:
        qo, ko = out
        at = (_given(qo, "out[0]", q.shape, io, device), _given(ko, "out[1]", k.shape, io, device))
    st = _library().ssm_qk_norm_rotate_fwd(*args, *at, _raw_stream(device))
    if st:
        _check(st, "ssm_qk_norm_rotate_fwd")
    _written(qo, ko)
    return qo, ko


def qk_norm_rotate_bwd(q, k, cos, sin, positions=None, q_weight=None, k_weight=None, *, dq_out,
                       dk_out, eps: float = 1e-6, interleaved: bool = False,
                       need_dweight: bool = True, workspace=None):
    """Gradients of ``qk_norm_rotate`` for upstream dq_out and dk_out.  Returns
    a dict: dq, dk in the I/O dtype; dq_weight, dk_weight [dim] float32 (None
    where the weight is None or without need_dweight)."""
    if workspace is None:
        r = _outputs(_native().rotate_bwd(
            _entry["ssm_qk_norm_rotate_bwd"], _entry["ssm_qk_norm_rotate_bwd_workspace_bytes"], q,
            k, cos, sin, positions, q_weight, k_weight, eps, interleaved, dq_out, dk_out,
            need_dweight), "ssm_qk_norm_rotate_bwd")
        if r is not None:
            return dict(zip(("dq", "dk", "dq_weight", "dk_weight"), r))
    args = _rotate_args(q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved)
    device, io = q.device, q.dtype
    dqo = _strided(dq_out, "dq_out", q.shape, io, device)
    dko = _strided(dk_out, "dk_out", k.shape, io, device)

    def dweight(w):
        return torch.empty_like(w) if w is not None and need_dweight else None
    g = {"dq": torch.empty_like(q, memory_format=_WHOLE),
         "dk": torch.empty_like(k, memory_format=_WHOLE),
         "dq_weight": dweight(q_weight), "dk_weight": dweight(k_weight)}
    lib = _library()
    nbytes = 0
    if g["dq_weight"] is not None or g["dk_weight"] is not None:
        nbytes = lib.ssm_qk_norm_rotate_bwd_workspace_bytes(args[0], args[2], args[3], args[4])
    ws, ws_bytes, keep = _workspace(nbytes, workspace, device)
    st = lib.ssm_qk_norm_rotate_bwd(*args, *dqo, *dko, _addr(g["dq"]), _addr(g["dk"]),
                                    _addr(g["dq_weight"]), _addr(g["dk_weight"]), ws, ws_bytes,
                                    _raw_stream(device))
    if st:
        _check(st, "ssm_qk_norm_rotate_bwd")
    return g


class QkNormRotate(torch.autograd.Function):
    """Autograd wrapper of ``qk_norm_rotate``: apply(q, k, cos, sin, positions,
    q_weight, k_weight, eps, interleaved) -> (q, k).  Differentiable once; cos
    and sin have no gradient."""

    @staticmethod
    def forward(ctx, q, k, cos, sin, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                interleaved=False):
        ctx.save_for_backward(q, k, cos, sin, positions, q_weight, k_weight)
        ctx.opts = (eps, interleaved)
        return qk_norm_rotate(q, k, cos, sin, positions, q_weight, k_weight, eps=eps,
                              interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        if any(ctx.needs_input_grad[2:4]):
            raise ValueError("cos and sin have no gradient: detach them")
        q, k, cos, sin, positions, q_weight, k_weight = ctx.saved_tensors
        eps, interleaved = ctx.opts
        g = qk_norm_rotate_bwd(q, k, cos, sin, positions, q_weight, k_weight,
                               dq_out=_as_operand(dq_out), dk_out=_as_operand(dk_out), eps=eps,
                               interleaved=interleaved,
                               need_dweight=any(ctx.needs_input_grad[5:7]))
        return (g["dq"], g["dk"], None, None, None, g["dq_weight"], g["dk_weight"], None, None)


def _delta_args(q, k, v, log_decay, beta, h0, cu_seqlens):
    """Checked operands of the whole-sequence calls: (shape of v without its
    channels, sizes for the workspace, arguments up to beta, state shape, h0)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{n} must be a torch.Tensor")
    nd = 4 if cu_seqlens is None else 3
    if q.dim() != nd or k.dim() != nd or v.dim() != nd:
        raise ValueError("q, k and v must be [batch, seqlen, heads, dim] tensors, or [tokens, "
                         "heads, dim] with cu_seqlens")
    device = q.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    *lead, kheads, kdim = q.shape
    heads, vdim = v.shape[-2:]
    if cu_seqlens is None:
        batch, seqlen = lead
        cu = None
    else:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 \
                or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a [sequences + 1] tensor")
        cu = _given(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, device)
        batch, seqlen = cu_seqlens.numel() - 1, lead[0]
        if batch == 0 and seqlen > 0:
            raise ValueError("tokens without a sequence")
    if heads and (kheads == 0 or heads % kheads):
        raise ValueError("v's heads must split evenly over those of q and k")
    io = q.dtype
    code = _io_code(io)
    state = (batch, heads, vdim, kdim)
    sizes = (batch, seqlen, cu is not None, heads, kheads, kdim, vdim, code)
    args = (batch, seqlen, cu, heads, kheads, kdim, vdim, code,
            q.data_ptr(), _token_stride(q, "q", q.shape),
            *_strided(k, "k", q.shape, io, device),
            *_strided(v, "v", (*lead, heads, vdim), io, device),
            _given(log_decay, "log_decay", (*lead, heads), torch.float32, device),
            _given(beta, "beta", (*lead, heads), io, device))
    return (*lead, heads), sizes, args, state, _optional(h0, "h0", state, torch.float32, device)


def gated_delta(q, k, v, log_decay, beta, h0=None, *, scale: float = 1.0, cu_seqlens=None,
                return_last_state=False, out=None, workspace=None):
    """Gated delta rule (``ssm_delta_fwd``): r_t = v_t - a_t S_{t-1} k_t, S_t =
    a_t S_{t-1} + beta_t r_t k_t^T, o_t = scale S_t q_t with a_t =
    exp(log_decay_t).  q, k [batch, L, key_heads, kdim], v [batch, L, heads,
    vdim] (float32 or bfloat16; tokens may be strided; heads / key_heads value
    heads share a key head), log_decay [batch, L, heads] float32, beta [batch,
    L, heads] of q's type; or all without the batch dimension and with
    ``cu_seqlens`` (int32 [sequences + 1] on the device, from 0 to the number of
    tokens) for packed sequences; h0 [sequences, heads, vdim, kdim] float32.
    kdim up to 128, vdim up to 256, multiples of 8.  Returns o [batch, L, heads,
    vdim] (and the final state when ``return_last_state``)."""
    if out is None and workspace is None:
        r = _outputs(_native().delta_fwd(
            _entry["ssm_delta_fwd"], _entry["ssm_delta_fwd_workspace_bytes"], q, k, v, log_decay,
            beta, h0, cu_seqlens, scale, return_last_state), "ssm_delta_fwd")
        if r is not None:
            return r if return_last_state else r[0]
    lead, sizes, args, state, h0_at = _delta_args(q, k, v, log_decay, beta, h0, cu_seqlens)
    device = q.device
    shape = (*lead, v.shape[-1])
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=device)
    o_at = _given(out, "out", shape, q.dtype, device)
    h_last = torch.empty(state, dtype=torch.float32, device=device) if return_last_state else None
    lib = _library()
    ws, ws_bytes, keep = _workspace(lib.ssm_delta_fwd_workspace_bytes(*sizes), workspace, device)
    st = lib.ssm_delta_fwd(*args, scale, h0_at, o_at, _addr(h_last), ws, ws_bytes,
                           _raw_stream(device))
    if st:
        _check(st, "ssm_delta_fwd")
    _written(out)
    return (out, h_last) if return_last_state else out


def gated_delta_bwd(q, k, v, log_decay, beta, h0=None, *, dy, dh_last=None, scale: float = 1.0,
                    cu_seqlens=None, need_dh0: bool = True, workspace=None):
    """Gradients of ``gated_delta`` for upstream dy (and dh_last).  Returns a
    dict: dq, dk (summed over the value heads that share them), dv and dbeta in
    the I/O dtype, dlog_decay and dh0 (None unless need_dh0) in float32.
    Gradients of tokens that no packed sequence holds are not written."""
    if workspace is None:
        r = _outputs(_native().delta_bwd(
            _entry["ssm_delta_bwd"], _entry["ssm_delta_bwd_workspace_bytes"], q, k, v, log_decay,
            beta, h0, cu_seqlens, scale, dy, dh_last, need_dh0), "ssm_delta_bwd")
        if r is not None:
            return dict(zip(("dq", "dk", "dv", "dlog_decay", "dbeta", "dh0"), r))
    lead, sizes, args, state, h0_at = _delta_args(q, k, v, log_decay, beta, h0, cu_seqlens)
    device, io = q.device, q.dtype
    dy_at = _strided(dy, "dy", (*lead, v.shape[-1]), io, device)
    dh_at = _optional(dh_last, "dh_last", state, torch.float32, device)
    g = {"dq": torch.empty_like(q, memory_format=_WHOLE),
         "dk": torch.empty_like(k, memory_format=_WHOLE),
         "dv": torch.empty_like(v, memory_format=_WHOLE),
         "dlog_decay": torch.empty_like(log_decay), "dbeta": torch.empty_like(beta),
         "dh0": torch.empty(state, dtype=torch.float32, device=device) if need_dh0 else None}
    lib = _library()
    ws, ws_bytes, keep = _workspace(lib.ssm_delta_bwd_workspace_bytes(*sizes), workspace, device)
    st = lib.ssm_delta_bwd(*args, scale, h0_at, *dy_at, dh_at, _addr(g["dq"]), _addr(g["dk"]),
                           _addr(g["dv"]), _addr(g["dlog_decay"]), _addr(g["dbeta"]),
                           _addr(g["dh0"]), ws, ws_bytes, _raw_stream(device))
    if st:
        _check(st, "ssm_delta_bwd")
    return g


def gated_delta_step(h, q, k, v, log_decay, beta, *, scale: float = 1.0, slots=None, out=None):
    """One token of ``gated_delta`` per row on resident states
    (``ssm_delta_step``).  h [nslots, heads, vdim, kdim] float32, updated in
    place; q, k [batch, key_heads, kdim], v [batch, heads, vdim]; log_decay
    [batch, heads] float32, beta [batch, heads] of q's type; ``slots`` int32
    [batch] names each row's state (None: row b uses slot b; a row with a slot
    outside [0, nslots) answers zeros).  Returns o [batch, heads, vdim]."""
    if out is None:
        r = _outputs(_native().delta_step(_entry["ssm_delta_step"], h, q, k, v, log_decay, beta,
                                          scale, slots), "ssm_delta_step")
        if r is not None:
            return r[0]
    if not isinstance(h, torch.Tensor) or h.dim() != 4:
        raise ValueError("h must be a [nslots, heads, vdim, kdim] tensor")
    device = h.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q, k and v must be [batch, heads, dim] tensors")
    nslots, heads, vdim, kdim = h.shape
    batch, kheads = q.shape[0], q.shape[1]
    if heads and (kheads == 0 or heads % kheads):
        raise ValueError("v's heads must split evenly over those of q and k")
    if slots is None and nslots < batch:
        raise ValueError(f"h holds {nslots} states for {batch} rows")
    io = q.dtype
    shape = (batch, heads, vdim)
    if out is None:
        out = torch.empty(shape, dtype=io, device=device)
    st = _library().ssm_delta_step(
        batch, nslots, _optional(slots, "slots", (batch,), torch.int32, device), heads, kheads,
        kdim, vdim, _io_code(io), _given(h, "h", h.shape, torch.float32, device),
        *_strided(q, "q", (batch, kheads, kdim), io, device),
        *_strided(k, "k", (batch, kheads, kdim), io, device),
        *_strided(v, "v", (batch, heads, vdim), io, device),
        _given(log_decay, "log_decay", (batch, heads), torch.float32, device),
        _given(beta, "beta", (batch, heads), io, device), scale,
        _given(out, "out", shape, io, device), _raw_stream(device))
    if st:
        _check(st, "ssm_delta_step")
    _written(h, out)
    return out


class GatedDelta(torch.autograd.Function):
    """Autograd wrapper of ``gated_delta``: apply(q, k, v, log_decay, beta, h0,
    scale, cu_seqlens) -> (o, h_last); h0 and cu_seqlens may be None.
    Differentiable once; scale is a number, without a gradient."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, beta, h0=None, scale=1.0, cu_seqlens=None):
        o, h_last = gated_delta(q, k, v, log_decay, beta, h0, scale=scale, cu_seqlens=cu_seqlens,
                                return_last_state=True)
        ctx.save_for_backward(q, k, v, log_decay, beta, h0, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        if any(ctx.needs_input_grad[6:7]):
            raise ValueError("scale has no gradient: detach it, or scale q")
        q, k, v, log_decay, beta, h0, cu_seqlens = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        g = gated_delta_bwd(q, k, v, log_decay, beta, h0, dy=_as_operand(dy),
                            dh_last=None if dh_last is None else _as_operand(dh_last),
                            scale=ctx.scale, cu_seqlens=cu_seqlens,
                            need_dh0=h0 is not None and ctx.needs_input_grad[5])
        return (g["dq"], g["dk"], g["dv"], g["dlog_decay"], g["dbeta"], g["dh0"], None, None)


def _rows(t, name, shape, dtype, device):
    """Address of a [..., dim] tensor whose rows are contiguous and evenly
    spaced, and the elements between them."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    dim = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), dim
    if t.stride(-1) != 1 and dim > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    step, rows = None, 1  # of the dimensions from the last one on
    for n, s in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != rows * step:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        rows *= n
    return t.data_ptr(), dim if step is None else step


def _norm_args(x, weight):
    """Checked (rows, dim, dtype code, x's address and stride, weight's address)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a [..., dim] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    dim = x.shape[-1]
    code = _io_code(x.dtype)
    return (x.numel() // dim if dim else 0, dim, code, *_rows(x, "x", x.shape, x.dtype, device),
            _optional(weight, "weight", (dim,), torch.float32, device))


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, out=None):
    """Layer norm over the last dimension (``ssm_layer_norm_fwd``): x [..., dim]
    float32 or bfloat16, rows evenly spaced; weight, bias [dim] float32 or None.
    dim up to 16384.  Returns a contiguous tensor of x's shape."""
    if out is None:
        r = _outputs(_native().norm_fwd(_entry["ssm_layer_norm_fwd"], x, weight, bias, eps),
                     "ssm_layer_norm_fwd")
        if r is not None:
            return r[0]
    *args, w_at = _norm_args(x, weight)
    device = x.device
    b_at = _optional(bias, "bias", (x.shape[-1],), torch.float32, device)
    if out is None:
        out = torch.empty_like(x, memory_format=_WHOLE)
    st = _library().ssm_layer_norm_fwd(*args, w_at, b_at, eps,
                                       _given(out, "out", x.shape, x.dtype, device),
                                       _raw_stream(device))
    if st:
        _check(st, "ssm_layer_norm_fwd")
    _written(out)
    return out


def layer_norm_bwd(x, weight=None, *, dy, eps: float = 1e-5, need_dweight: bool = True,
                   need_dbias: bool = True, workspace=None):
    """Gradients of ``layer_norm`` for upstream dy (rows evenly spaced).  Returns
    a dict: dx in the I/O dtype; dweight, dbias [dim] float32, summed over the
    rows (None without need_dweight, need_dbias)."""
    if workspace is None:
        r = _outputs(_native().norm_bwd(
            _entry["ssm_layer_norm_bwd"], _entry["ssm_layer_norm_bwd_workspace_bytes"], x, weight,
            dy, eps, need_dweight, need_dbias), "ssm_layer_norm_bwd")
        if r is not None:
            return dict(zip(("dx", "dweight", "dbias"), r))
    *args, w_at = _norm_args(x, weight)
    device, dim = x.device, x.shape[-1]
    dy_at = _rows(dy, "dy", x.shape, x.dtype, device)

    def sums(needed):
        return torch.empty(dim, dtype=torch.float32, device=device) if needed else None
    g = {"dx": torch.empty_like(x, memory_format=_WHOLE), "dweight": sums(need_dweight),
         "dbias": sums(need_dbias)}
    lib = _library()
    nbytes = 0
    if need_dweight or need_dbias:
        nbytes = lib.ssm_layer_norm_bwd_workspace_bytes(*args[:3])
    ws, ws_bytes, keep = _workspace(nbytes, workspace, device)
    st = lib.ssm_layer_norm_bwd(*args, w_at, eps, *dy_at, _addr(g["dx"]), _addr(g["dweight"]),
                                _addr(g["dbias"]), ws, ws_bytes, _raw_stream(device))
    if st:
        _check(st, "ssm_layer_norm_bwd")
    return g


class LayerNorm(torch.autograd.Function):
    """Autograd wrapper of ``layer_norm``: apply(x, weight, bias, eps) -> y;
    weight and bias may be None.  Differentiable once."""

    @staticmethod
    def forward(ctx, x, weight=None, bias=None, eps=1e-5):
        ctx.save_for_backward(x, weight)
        ctx.eps = eps
        return layer_norm(x, weight, bias, eps=eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight = ctx.saved_tensors
        g = layer_norm_bwd(x, weight, dy=dy.contiguous(), eps=ctx.eps,
                           need_dweight=ctx.needs_input_grad[1], need_dbias=ctx.needs_input_grad[2])
        return g["dx"], g["dweight"], g["dbias"], None
