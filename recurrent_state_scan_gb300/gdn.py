"""Thin Python binding of libgdn's C ABI (argument marshalling only).

Every step of the scan runs in libgdn's CUDA kernels; PyTorch only supplies
device memory and the stream.  The entry points keep the C names:
``gdn_prefill``, ``gdn_decode_step``, ``gdn_prefill_workspace_bytes``,
``gdn_last_device_status``, ``gdn_status_string``.  If the library cannot be
loaded every call raises -- there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

from . import _build

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED = 0, 1, 2
GDN_ERR_CUDA, GDN_ERR_DEVICE_CHECK, GDN_ERR_TIMEOUT = 3, 4, 5
GDN_F32, GDN_BF16, GDN_F16 = 0, 1, 2
_DTYPE_CODE = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float16: GDN_F16}

# Every symbol include/gdn.h declares.
EXPORTS = ("gdn_prefill_workspace_bytes", "gdn_prefill", "gdn_decode_step",
           "gdn_prefill_plan", "gdn_last_device_status", "gdn_status_string",
           "gdn_last_error_message", "gdn_prefill_noalloc", "gdn_decode_step_slots",
           "gdn_scan_window", "gdn_scan_variant", "gdn_causal_conv", "gdn_causal_conv_slots",
           "gdn_gated_rmsnorm", "gdn_set_wait_budget", "gdn_decode_layer", "gdn_prefill_variant",
           "gdn_prefill_norm", "gdn_prefill_variant_workspace_bytes", "gdn_prefill_variant_plan",
           "gdn_prefill_layer", "gdn_prefill_layer_workspace_bytes", "gdn_ssm_prefill_workspace_bytes",
           "gdn_ssm_prefill", "gdn_ssm_prefill_plan", "gdn_ssm_decode", "gdn_rotary", "gdn_rotary_frequencies",
           "gdn_diag_kept_bytes", "gdn_diag_prefill_workspace_bytes", "gdn_diag_prefill", "gdn_diag_backward_workspace_bytes", "gdn_diag_backward",
           "gdn_diag_decode", "gdn_checkpoint_pack", "gdn_checkpoint_unpack")
PATH_SIMT, PATH_TC, PATH_TC_TP = 1, 2, 3
# gdn_rule codes.
RULES = {"gated_delta": 0, "delta": 1, "gated": 2, "linear": 3}
# gdn_activation codes.
ACTIVATIONS = {"none": 0, "silu": 1, "swish": 1, "sigmoid": 2}
# gdn_rotary_kind codes.
ROTARY_KINDS = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "wavelength": 4}
# gdn_diag_gate, gdn_diag_weighting and gdn_diag_keep codes.
DIAG_GATES = {"softplus": 0, "sigmoid": 1}
DIAG_WEIGHTINGS = {"plain": 0, "complement": 1, "norm": 2}
DIAG_KEEPS = {None: 0, "states": 1, "8bit": 2}
# Channels that share a step of the 8-bit codes.
CHECKPOINT_BLOCK = 64


class GdnShape(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seqlen", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("h_qk", ctypes.c_int32), ("h_v", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32)]


class GdnVariant(ctypes.Structure):
    _fields_ = [("rule", ctypes.c_int32), ("decay_per_key", ctypes.c_int32),
                ("beta_shared", ctypes.c_int32)]


class GdnConvShape(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int32),
                ("kernel", ctypes.c_int32), ("dilation", ctypes.c_int32),
                ("channels_last", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("state_window", ctypes.c_int32)]


class GdnLayerParams(ctypes.Structure):
    _fields_ = [("conv_kernel", ctypes.c_int32), ("conv_activation", ctypes.c_int32),
                ("norm_activation", ctypes.c_int32), ("norm_epsilon", ctypes.c_float)]


class GdnSsmShape(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seqlen", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("d_state", ctypes.c_int32),
                ("xbc_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("z_stride", ctypes.c_int64)]


class GdnSsmParams(ctypes.Structure):
    _fields_ = [("conv_kernel", ctypes.c_int32), ("conv_activation", ctypes.c_int32),
                ("dt_min", ctypes.c_float), ("dt_max", ctypes.c_float)]


class GdnRotaryShape(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seqlen", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("rot_offset", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("scale", ctypes.c_float)] + \
               [(name, ctypes.c_int64) for name in (
                   "q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                   "q_out_row_stride", "q_out_head_stride", "k_out_row_stride", "k_out_head_stride")]


class GdnRotaryScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("trained_length", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double)]


class GdnDiagShape(ctypes.Structure):
    _fields_ = [("io_dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seqlen", ctypes.c_int64), ("num_seqs", ctypes.c_int32),
                ("channels", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("weighting", ctypes.c_int32), ("input_gate", ctypes.c_int32),
                ("keep", ctypes.c_int32)] + \
               [(name, ctypes.c_int64) for name in (
                   "x_stride", "a_stride", "b_stride", "y_stride", "dx_stride", "da_stride", "db_stride")]


class GdnDiagKept(NamedTuple):
    """What gdn_diag_prefill keeps for gdn_diag_backward: the buffer, and the call that it belongs to."""
    data: torch.Tensor
    io: torch.dtype
    batch: int
    seqlen: int
    num_seqs: int
    channels: int
    gate: str
    weighting: str
    input_gate: bool
    keep: str


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libgdn.so (building it first if allowed).  Raises if unavailable."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB) or (build_if_missing and not _build.up_to_date()):
        if not build_if_missing:
            raise GdnError(GDN_ERR_CUDA, f"libgdn is not built ({_build.LIB})")
        _build.build()
    lib = ctypes.CDLL(_build.LIB)
    P = ctypes.c_void_p
    S = ctypes.POINTER(GdnShape)
    lib.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_prefill_workspace_bytes.argtypes = [S]
    lib.gdn_prefill.restype = ctypes.c_int
    lib.gdn_prefill.argtypes = [S, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P,
                                ctypes.c_size_t, P]
    lib.gdn_scan_window.restype = ctypes.c_int
    lib.gdn_scan_window.argtypes = [S, P, P, P, P, P, P, P, P, ctypes.c_float, P, P,
                                    ctypes.c_int32, P]
    CS = ctypes.POINTER(GdnConvShape)
    lib.gdn_causal_conv.restype = ctypes.c_int
    lib.gdn_causal_conv.argtypes = [CS, P, P, P, P, P, P, P]
    lib.gdn_causal_conv_slots.restype = ctypes.c_int
    lib.gdn_causal_conv_slots.argtypes = [CS, P, P, P, P, ctypes.c_int64, P, P, P]
    lib.gdn_gated_rmsnorm.restype = ctypes.c_int
    lib.gdn_gated_rmsnorm.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, P, P, P,
                                      ctypes.c_float, ctypes.c_int32, P, P]
    lib.gdn_scan_variant.restype = ctypes.c_int
    lib.gdn_scan_variant.argtypes = [S, ctypes.POINTER(GdnVariant), P, P, P, P, P, P, P, P, P,
                                     ctypes.c_float, P, P, P]
    lib.gdn_decode_step_slots.restype = ctypes.c_int
    lib.gdn_decode_step_slots.argtypes = [S, P, P, P, P, P, P, P, P, ctypes.c_int64, P,
                                          ctypes.c_float, P, P]
    lib.gdn_prefill_noalloc.restype = ctypes.c_int
    lib.gdn_prefill_noalloc.argtypes = [S, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [S, P, P, P, P, P, P, P, P, ctypes.c_float, P, P]
    lib.gdn_prefill_plan.restype = ctypes.c_int
    lib.gdn_prefill_plan.argtypes = [S, ctypes.POINTER(ctypes.c_int32),
                                     ctypes.POINTER(ctypes.c_int32)]
    lib.gdn_last_device_status.restype = ctypes.c_int
    lib.gdn_last_device_status.argtypes = [P]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_last_error_message.restype = ctypes.c_char_p
    lib.gdn_last_error_message.argtypes = []
    lib.gdn_set_wait_budget.restype = ctypes.c_int
    lib.gdn_set_wait_budget.argtypes = [ctypes.c_int64]
    lib.gdn_prefill_variant.restype = ctypes.c_int
    lib.gdn_prefill_variant.argtypes = [S, ctypes.POINTER(GdnVariant), P, P, P, P, P, P, P, P, P,
                                        ctypes.c_float, P, P, P, ctypes.c_size_t, P]
    lib.gdn_prefill_variant_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_prefill_variant_workspace_bytes.argtypes = [S, ctypes.POINTER(GdnVariant)]
    lib.gdn_prefill_variant_plan.restype = ctypes.c_int
    lib.gdn_prefill_variant_plan.argtypes = [S, ctypes.POINTER(GdnVariant), ctypes.POINTER(ctypes.c_int32),
                                             ctypes.POINTER(ctypes.c_int32)]
    lib.gdn_prefill_norm.restype = ctypes.c_int
    lib.gdn_prefill_norm.argtypes = [S, P, P, P, P, P, P, P, P, P, ctypes.c_float, P, P,
                                     ctypes.c_float, ctypes.c_int32, ctypes.c_int32, P, P, P,
                                     ctypes.c_size_t, P]
    SS, SP = ctypes.POINTER(GdnSsmShape), ctypes.POINTER(GdnSsmParams)
    lib.gdn_ssm_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_ssm_prefill_workspace_bytes.argtypes = [SS, SP]
    lib.gdn_ssm_prefill.restype = ctypes.c_int
    lib.gdn_ssm_prefill.argtypes = [SS, SP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.gdn_ssm_prefill_plan.restype = ctypes.c_int
    lib.gdn_ssm_prefill_plan.argtypes = [SS, SP, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.gdn_ssm_decode.restype = ctypes.c_int
    lib.gdn_ssm_decode.argtypes = [SS, SP, P, P, P, P, P, P, P, P, P, P, ctypes.c_int64, P, P, P]
    lib.gdn_rotary.restype = ctypes.c_int
    lib.gdn_rotary.argtypes = [ctypes.POINTER(GdnRotaryShape), P, P, P, P, P, P, P, P]
    lib.gdn_rotary_frequencies.restype = ctypes.c_int
    lib.gdn_rotary_frequencies.argtypes = [ctypes.POINTER(GdnRotaryScaling), ctypes.c_int32, P,
                                           ctypes.POINTER(ctypes.c_float)]
    DS = ctypes.POINTER(GdnDiagShape)
    lib.gdn_diag_kept_bytes.restype = ctypes.c_size_t
    lib.gdn_diag_kept_bytes.argtypes = [DS]
    lib.gdn_diag_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_diag_prefill_workspace_bytes.argtypes = [DS]
    lib.gdn_diag_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_diag_backward_workspace_bytes.argtypes = [DS]
    lib.gdn_diag_prefill.restype = ctypes.c_int
    lib.gdn_diag_prefill.argtypes = [DS, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P, ctypes.c_size_t, P]
    lib.gdn_diag_backward.restype = ctypes.c_int
    lib.gdn_diag_backward.argtypes = [DS, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P, P, P, P, P, P, P, P, P, P,
                                      ctypes.c_size_t, P]
    lib.gdn_diag_decode.restype = ctypes.c_int
    lib.gdn_diag_decode.argtypes = [DS, P, P, P, P, P, P, P, ctypes.c_int64, P, P, P]
    lib.gdn_checkpoint_pack.restype = ctypes.c_int
    lib.gdn_checkpoint_pack.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, P, ctypes.c_int64, P, P, P]
    lib.gdn_checkpoint_unpack.restype = ctypes.c_int
    lib.gdn_checkpoint_unpack.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, P, P, P, ctypes.c_int64, P]
    lib.gdn_decode_layer.restype = ctypes.c_int
    lib.gdn_decode_layer.argtypes = [S, ctypes.POINTER(GdnLayerParams), P, P, P, P, P, P, P, P, P,
                                     P, ctypes.c_float, P, P, P, P]
    lib.gdn_prefill_layer.restype = ctypes.c_int
    lib.gdn_prefill_layer.argtypes = [S, ctypes.POINTER(GdnLayerParams), P, P, P, P, P, P, P, P, P, P, P,
                                      ctypes.c_float, P, P, P, P, ctypes.c_int32, P, ctypes.c_size_t, P]
    lib.gdn_prefill_layer_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_prefill_layer_workspace_bytes.argtypes = [S]
    _lib = lib
    return lib


def status_name(status: int) -> str:
    try:
        return load().gdn_status_string(int(status)).decode()
    except Exception:  # the name is only cosmetic
        return f"status {status}"


def _check(status: int):
    if status != GDN_OK:
        raise GdnError(status, load().gdn_last_error_message().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need_cuda(name: str, t: torch.Tensor, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be {dtype}, got {t.dtype}")


def make_shape(io_dtype: int, batch: int, seqlen: int, num_seqs: int, h_qk: int, h_v: int,
               d_k: int, d_v: int) -> GdnShape:
    return GdnShape(io_dtype, batch, seqlen, num_seqs, h_qk, h_v, d_k, d_v)


def _shape_of(q, v, cu_seqlens) -> GdnShape:
    if q.dim() != 4 or v.dim() != 4:
        raise GdnError(GDN_ERR_INVALID_ARG, "q and v must be [B, T, H, D]")
    B, T, h_qk, d_k = q.shape
    h_v, d_v = v.shape[2], v.shape[3]
    if q.dtype not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unsupported io dtype {q.dtype}")
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    return make_shape(_DTYPE_CODE[q.dtype], B, T, n, h_qk, h_v, d_k, d_v)


def gdn_prefill_workspace_bytes(shape: GdnShape) -> int:
    return int(load().gdn_prefill_workspace_bytes(ctypes.byref(shape)))


def gdn_prefill(q, k, v, a, b, A_log, dt_bias, state_in=None, cu_seqlens=None,
                scale: float = 0.0, *, o=None, state_out=None, workspace=None, stream=None):
    """Run the gated delta rule over whole sequences; returns (o, state_out).

    q, k [B,T,h_qk,d_k]; v [B,T,h_v,d_v]; a, b [B,T,h_v] (all one io dtype);
    A_log, dt_bias [h_v] fp32; state_in [N,h_v,d_k,d_v] fp32 or None;
    cu_seqlens int32 [N+1] on the device (then B must be 1) or None.
    """
    lib = load()
    shape = _shape_of(q, v, cu_seqlens)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need_cuda(name, t, dt)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    if tuple(k.shape) != tuple(q.shape) or tuple(a.shape) != tuple(v.shape[:3]) or \
            tuple(b.shape) != tuple(a.shape):
        raise GdnError(GDN_ERR_INVALID_ARG, "k must match q, and a, b must be [B, T, h_v]")
    if tuple(A_log.shape) != (shape.h_v,) or tuple(dt_bias.shape) != (shape.h_v,):
        raise GdnError(GDN_ERR_INVALID_ARG, "A_log and dt_bias must be [h_v]")
    st_shape = (shape.num_seqs, shape.h_v, shape.d_k, shape.d_v)
    if state_in is not None:
        _need_cuda("state_in", state_in, torch.float32)
        if tuple(state_in.shape) != st_shape:
            raise GdnError(GDN_ERR_INVALID_ARG, f"state_in must be {st_shape}")
    if cu_seqlens is not None:
        _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    if o is None:
        o = torch.empty(v.shape, dtype=dt, device=v.device)
    else:
        _need_cuda("o", o, dt)
    if state_out is None:
        state_out = torch.empty(st_shape, dtype=torch.float32, device=v.device)
    else:
        _need_cuda("state_out", state_out, torch.float32)
    need = int(lib.gdn_prefill_workspace_bytes(ctypes.byref(shape)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_prefill(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                           _ptr(A_log), _ptr(dt_bias), _ptr(state_in), _ptr(cu_seqlens),
                           float(scale), _ptr(o), _ptr(state_out), _ptr(workspace), ws_bytes,
                           _stream(stream)))
    return o, state_out


# Size of the library's fixed scratch array behind gdn_prefill_noalloc.
PREFILL_NOALLOC_SCRATCH_BYTES = 96 * 1024 * 1024



def gdn_prefill_norm(q, k, v, a, b, A_log, dt_bias, state_in=None, cu_seqlens=None,
                     scale: float = 0.0, *, norm_scale, gate, eps: float = 1e-6,
                     activation: str = "silu", fuse: bool = False, y=None, state_out=None,
                     workspace=None, stream=None):
    """gdn_prefill, then the gated RMS norm of o over each d_v row; returns (y, state_out).

    norm_scale [d_v] and gate (o's shape) in the io dtype; y has o's shape.  fuse: run the
    norm in the tensor-core scan's readout (o never stored) where the path allows; by
    default the norm is a second launch, in place on y."""
    lib = load()
    shape = _shape_of(q, v, cu_seqlens)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("gate", gate),
                    ("norm_scale", norm_scale)):
        _need_cuda(name, t, dt)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    if tuple(k.shape) != tuple(q.shape) or tuple(a.shape) != tuple(v.shape[:3]) or \
            tuple(b.shape) != tuple(a.shape):
        raise GdnError(GDN_ERR_INVALID_ARG, "k must match q, and a, b must be [B, T, h_v]")
    if tuple(gate.shape) != tuple(v.shape) or tuple(norm_scale.shape) != (shape.d_v,):
        raise GdnError(GDN_ERR_INVALID_ARG, "gate must match v, norm_scale must be [d_v]")
    if activation not in ("silu", "swish", "sigmoid"):
        raise GdnError(GDN_ERR_INVALID_ARG, "activation is silu or sigmoid")
    st_shape = (shape.num_seqs, shape.h_v, shape.d_k, shape.d_v)
    if state_in is not None:
        _need_cuda("state_in", state_in, torch.float32)
        if tuple(state_in.shape) != st_shape:
            raise GdnError(GDN_ERR_INVALID_ARG, f"state_in must be {st_shape}")
    if cu_seqlens is not None:
        _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    if y is None:
        y = torch.empty(v.shape, dtype=dt, device=v.device)
    else:
        _need_cuda("y", y, dt)
    if state_out is None:
        state_out = torch.empty(st_shape, dtype=torch.float32, device=v.device)
    else:
        _need_cuda("state_out", state_out, torch.float32)
    need = int(lib.gdn_prefill_workspace_bytes(ctypes.byref(shape)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_prefill_norm(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                                _ptr(A_log), _ptr(dt_bias), _ptr(state_in), _ptr(cu_seqlens),
                                float(scale), _ptr(norm_scale), _ptr(gate), float(eps),
                                ACTIVATIONS[activation], int(bool(fuse)), _ptr(y), _ptr(state_out),
                                _ptr(workspace), ws_bytes, _stream(stream)))
    return y, state_out


def gdn_prefill_noalloc(q, k, v, a, b, A_log, dt_bias, state_in, cu_seqlens, scale: float,
                        *, o, state_out, stream=None):
    """gdn_prefill for callers that may not allocate device memory: the outputs are
    caller-provided and the tensor-core path's scratch is the library's fixed
    96 MiB array, shared by every call on the device (calls that overlap on the GPU
    race on it).  Shapes needing more scratch raise GDN_ERR_INVALID_ARG."""
    lib = load()
    shape = _shape_of(q, v, cu_seqlens)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("o", o)):
        _need_cuda(name, t, dt)
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias), ("state_out", state_out)):
        _need_cuda(name, t, torch.float32)
    if state_in is not None:
        _need_cuda("state_in", state_in, torch.float32)
    if cu_seqlens is not None:
        _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    st_shape = (shape.num_seqs, shape.h_v, shape.d_k, shape.d_v)
    if tuple(o.shape) != tuple(v.shape) or tuple(state_out.shape) != st_shape:
        raise GdnError(GDN_ERR_INVALID_ARG, f"o must be {tuple(v.shape)} and state_out {st_shape}")
    _check(lib.gdn_prefill_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                   _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(state_in),
                                   _ptr(cu_seqlens), float(scale), _ptr(o), _ptr(state_out),
                                   _stream(stream)))
    return o, state_out


def gdn_decode_step(q, k, v, a, b, A_log, dt_bias, state, scale: float = 0.0, *, o=None,
                    stream=None):
    """One token per sequence; ``state`` [B,h_v,d_k,d_v] fp32 is updated in place.

    q, k [B,1,h_qk,d_k]; v [B,1,h_v,d_v]; a, b [B,1,h_v].  Returns o [B,1,h_v,d_v].
    """
    lib = load()
    shape = _shape_of(q, v, None)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need_cuda(name, t, dt)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    _need_cuda("state", state, torch.float32)
    if tuple(state.shape) != (shape.batch, shape.h_v, shape.d_k, shape.d_v):
        raise GdnError(GDN_ERR_INVALID_ARG, "state must be [B, h_v, d_k, d_v]")
    if o is None:
        o = torch.empty(v.shape, dtype=dt, device=v.device)
    else:
        _need_cuda("o", o, dt)
    _check(lib.gdn_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                               _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(state), float(scale),
                               _ptr(o), _stream(stream)))
    return o


def gdn_prefill_plan(shape: GdnShape):
    """(path, launches per call) that gdn_prefill takes for ``shape``."""
    path, launches = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load().gdn_prefill_plan(ctypes.byref(shape), ctypes.byref(path),
                                   ctypes.byref(launches)))
    return path.value, launches.value


def gdn_prefill_variant_plan(shape: GdnShape, rule: str = "gated_delta", decay_per_key: bool = False,
                             beta_shared: bool = False):
    """(path, launches per call) that gdn_prefill_variant takes for ``shape`` with the
    workspace gdn_prefill_variant_workspace_bytes reports."""
    if rule not in RULES:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unknown rule {rule!r}")
    var = GdnVariant(RULES[rule], int(bool(decay_per_key)), int(bool(beta_shared)))
    path, launches = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load().gdn_prefill_variant_plan(ctypes.byref(shape), ctypes.byref(var), ctypes.byref(path),
                                           ctypes.byref(launches)))
    return path.value, launches.value


def gdn_prefill_layer_workspace_bytes(shape: GdnShape) -> int:
    """The workspace gdn_prefill_layer needs for ``shape`` (0 off the tensor-core shapes)."""
    return int(load().gdn_prefill_layer_workspace_bytes(ctypes.byref(shape)))


def gdn_prefill_variant_workspace_bytes(shape: GdnShape, rule: str = "gated_delta",
                                        decay_per_key: bool = False, beta_shared: bool = False) -> int:
    if rule not in RULES:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unknown rule {rule!r}")
    var = GdnVariant(RULES[rule], int(bool(decay_per_key)), int(bool(beta_shared)))
    return int(load().gdn_prefill_variant_workspace_bytes(ctypes.byref(shape), ctypes.byref(var)))


def shape_of_spec(spec, n_seq: int, total_tokens: int) -> GdnShape:
    io = {"f32": GDN_F32, "bf16": GDN_BF16, "f16": GDN_F16}[spec.io]
    if spec.lengths is not None or spec.varlen_range is not None:
        return make_shape(io, 1, total_tokens, n_seq, spec.h_qk, spec.h_v, spec.d_k, spec.d_v)
    return make_shape(io, spec.batch, spec.seqlen, spec.batch, spec.h_qk, spec.h_v, spec.d_k,
                      spec.d_v)


def _simt_only(spec) -> bool:
    """Specs that run the token-sequential kernel alone: decode and state windows (the
    rules, the shared beta and the per-key-dim decay of a prefill take gdn_prefill's path
    through gdn_prefill_variant)."""
    return bool(spec.decode or getattr(spec, "window", 0))


def gdn_set_wait_budget(cycles: int) -> None:
    """Test hook: cycles a bounded wait of the tensor-core prefill kernels may take before
    the CTA gives up (0: the default, about two seconds)."""
    _check(load().gdn_set_wait_budget(int(cycles)))


def launches_per_call(spec, n_seq: int = 0, total_tokens: int = 0) -> int:
    if _simt_only(spec):
        return 1
    return gdn_prefill_plan(shape_of_spec(spec, n_seq, total_tokens))[1]


def path_dtype(spec, n_seq: int = 0, total_tokens: int = 0) -> str:
    """Arithmetic type of the path: MMA operand type on the tensor-core path, else f32."""
    if _simt_only(spec):
        return "f32"
    path = gdn_prefill_plan(shape_of_spec(spec, n_seq, total_tokens))[0]
    return spec.io if path in (PATH_TC, PATH_TC_TP) else "f32"


def gdn_last_device_status(stream=None) -> int:
    """Synchronise, read and clear the device check word; returns the status code."""
    return int(load().gdn_last_device_status(_stream(stream)))


def gdn_status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def gdn_decode_step_slots(q, k, v, a, b, A_log, dt_bias, pool, slots, scale: float = 0.0, *,
                          o=None, stream=None):
    """One token per sequence against a pool of states: sequence b reads and updates
    ``pool[slots[b]]`` in place.  q, k [B,1,h_qk,d_k]; v [B,1,h_v,d_v]; a, b [B,1,h_v];
    pool [P,h_v,d_k,d_v] fp32; slots int32 [B] on the device.  Returns o [B,1,h_v,d_v]."""
    lib = load()
    shape = _shape_of(q, v, None)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need_cuda(name, t, dt)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    _need_cuda("pool", pool, torch.float32)
    _need_cuda("slots", slots, torch.int32)
    if pool.dim() != 4 or tuple(pool.shape[1:]) != (shape.h_v, shape.d_k, shape.d_v):
        raise GdnError(GDN_ERR_INVALID_ARG, "pool must be [P, h_v, d_k, d_v]")
    if tuple(slots.shape) != (shape.batch,):
        raise GdnError(GDN_ERR_INVALID_ARG, "slots must be [B]")
    if o is None:
        o = torch.empty(v.shape, dtype=dt, device=v.device)
    else:
        _need_cuda("o", o, dt)
    _check(lib.gdn_decode_step_slots(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                     _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(pool),
                                     int(pool.shape[0]), _ptr(slots), float(scale), _ptr(o),
                                     _stream(stream)))
    return o


def gdn_scan_window(q, k, v, a, b, A_log, dt_bias, state_in=None, scale: float = 0.0, *,
                    window_len: int, o=None, window=None, stream=None):
    """Run B sequences of T tokens and return (o, window): window[w] is the state after
    step T - window_len + w, with zero slabs first when T < window_len.
    q, k [B,T,h_qk,d_k]; v [B,T,h_v,d_v]; a, b [B,T,h_v]; state_in [B,h_v,d_k,d_v] or None;
    window [window_len, B, h_v, d_k, d_v] fp32."""
    lib = load()
    shape = _shape_of(q, v, None)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b)):
        _need_cuda(name, t, dt)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    st_shape = (shape.batch, shape.h_v, shape.d_k, shape.d_v)
    if state_in is not None:
        _need_cuda("state_in", state_in, torch.float32)
        if tuple(state_in.shape) != st_shape:
            raise GdnError(GDN_ERR_INVALID_ARG, f"state_in must be {st_shape}")
    if o is None:
        o = torch.empty(v.shape, dtype=dt, device=v.device)
    else:
        _need_cuda("o", o, dt)
    if window is None:
        window = torch.empty((int(window_len),) + st_shape, dtype=torch.float32, device=v.device)
    else:
        _need_cuda("window", window, torch.float32)
    _check(lib.gdn_scan_window(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                               _ptr(A_log), _ptr(dt_bias), _ptr(state_in), float(scale), _ptr(o),
                               _ptr(window), int(window_len), _stream(stream)))
    return o, window


def _variant_args(q, k, v, a, b, A_log, dt_bias, state_in, cu_seqlens, rule, decay_per_key,
                  beta_shared, o, state_out):
    """Validate a variant call; returns (shape, variant, o, state_out, the pointers a, b,
    A_log, dt_bias the rule reads)."""
    if rule not in RULES:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unknown rule {rule!r}")
    shape = _shape_of(q, v, cu_seqlens)
    dt = q.dtype
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, dt)
    if tuple(k.shape) != tuple(q.shape):
        raise GdnError(GDN_ERR_INVALID_ARG, "k must match q")
    lead = tuple(v.shape[:2])
    decay = rule in ("gated_delta", "gated")
    delta = rule in ("gated_delta", "delta")
    if decay:
        _need_cuda("a", a, dt)
        _need_cuda("A_log", A_log, torch.float32)
        _need_cuda("dt_bias", dt_bias, torch.float32)
        per = (shape.h_v, shape.d_k) if decay_per_key else (shape.h_v,)
        if tuple(a.shape) != lead + per or tuple(A_log.shape) != per or \
                tuple(dt_bias.shape) != per:
            raise GdnError(GDN_ERR_INVALID_ARG, f"a must be {lead + per}, A_log and dt_bias {per}")
    if delta:
        _need_cuda("b", b, dt)
        want = lead + ((1,) if beta_shared else (shape.h_v,))
        if tuple(b.shape) != want:
            raise GdnError(GDN_ERR_INVALID_ARG, f"b must be {want}")
    st_shape = (shape.num_seqs, shape.h_v, shape.d_k, shape.d_v)
    if state_in is not None:
        _need_cuda("state_in", state_in, torch.float32)
        if tuple(state_in.shape) != st_shape:
            raise GdnError(GDN_ERR_INVALID_ARG, f"state_in must be {st_shape}")
    if cu_seqlens is not None:
        _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    if o is None:
        o = torch.empty(v.shape, dtype=dt, device=v.device)
    else:
        _need_cuda("o", o, dt)
    if state_out is None:
        state_out = torch.empty(st_shape, dtype=torch.float32, device=v.device)
    else:
        _need_cuda("state_out", state_out, torch.float32)
    var = GdnVariant(RULES[rule], int(bool(decay_per_key)), int(bool(beta_shared)))
    gates = (_ptr(a if decay else None), _ptr(b if delta else None),
             _ptr(A_log if decay else None), _ptr(dt_bias if decay else None))
    return shape, var, o, state_out, gates


def gdn_scan_variant(q, k, v, a=None, b=None, A_log=None, dt_bias=None, state_in=None,
                     cu_seqlens=None, scale: float = 0.0, *, rule: str = "gated_delta",
                     decay_per_key: bool = False, beta_shared: bool = False, o=None,
                     state_out=None, stream=None):
    """gdn_prefill with another update rule ("gated_delta", "delta", "gated", "linear"),
    per-key-dim decay (a [B,T,h_v,d_k]; A_log, dt_bias [h_v,d_k]) or one beta for all
    heads (b [B,T,1]), on the token-sequential kernel.  a, A_log, dt_bias are unused (may
    be None) by rules without decay, b by rules without the delta term.  Returns
    (o, state_out); ``state_out`` may be ``state_in`` itself (an in-place update)."""
    lib = load()
    shape, var, o, state_out, gates = _variant_args(q, k, v, a, b, A_log, dt_bias, state_in,
                                                    cu_seqlens, rule, decay_per_key, beta_shared,
                                                    o, state_out)
    _check(lib.gdn_scan_variant(ctypes.byref(shape), ctypes.byref(var), _ptr(q), _ptr(k), _ptr(v),
                                *gates, _ptr(state_in), _ptr(cu_seqlens), float(scale), _ptr(o),
                                _ptr(state_out), _stream(stream)))
    return o, state_out


def gdn_prefill_variant(q, k, v, a=None, b=None, A_log=None, dt_bias=None, state_in=None,
                        cu_seqlens=None, scale: float = 0.0, *, rule: str = "gated_delta",
                        decay_per_key: bool = False, beta_shared: bool = False, o=None,
                        state_out=None, workspace=None, stream=None):
    """gdn_scan_variant on gdn_prefill's path: the chunked tensor-core prefill for 16-bit
    I/O at d_k = d_v = 128 (any rule, shared or per-head beta, per-key-dim decay), the
    token-sequential kernel for other shapes.  ``workspace`` defaults to
    gdn_prefill_variant_workspace_bytes; a per-key decay given less (down to
    gdn_prefill_workspace_bytes) runs the token-sequential kernel."""
    lib = load()
    shape, var, o, state_out, gates = _variant_args(q, k, v, a, b, A_log, dt_bias, state_in,
                                                    cu_seqlens, rule, decay_per_key, beta_shared,
                                                    o, state_out)
    need = int(lib.gdn_prefill_variant_workspace_bytes(ctypes.byref(shape), ctypes.byref(var)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.gdn_prefill_variant(ctypes.byref(shape), ctypes.byref(var), _ptr(q), _ptr(k), _ptr(v),
                                   *gates, _ptr(state_in), _ptr(cu_seqlens), float(scale), _ptr(o),
                                   _ptr(state_out), _ptr(workspace), ws_bytes, _stream(stream)))
    return o, state_out


# ---------------------------------------------------------------- neighbouring ops

def _conv_geometry(x, weight, channels_last: bool):
    if x.dim() != 3:
        raise GdnError(GDN_ERR_INVALID_ARG, "x must be [B, L, C] (or [B, C, L])")
    if x.dtype not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unsupported io dtype {x.dtype}")
    B = x.shape[0]
    L, C = (x.shape[1], x.shape[2]) if channels_last else (x.shape[2], x.shape[1])
    if weight.numel() == 0 or weight.numel() % C != 0 or weight.shape[0] != C:
        raise GdnError(GDN_ERR_INVALID_ARG, "weight must be [C, 1, K] or [C, K, 1]")
    return B, L, C, weight.numel() // C


def conv_state_shape(B: int, C: int, K: int, dilation: int = 1, channels_last: bool = True,
                     state_window: int = 0):
    carry = (K - 1) * dilation
    shape = (B, carry, C) if channels_last else (B, C, carry)
    return ((state_window,) + shape) if state_window else shape


def gdn_causal_conv(x, weight, bias=None, state_in=None, *, dilation: int = 1,
                    channels_last: bool = True, activation: str = "none",
                    state_window: int = 0, y=None, state_out=None, stream=None):
    """Causal depthwise convolution with a carried state; returns (y, state_out).

    x [B, L, C] (channels_last) or [B, C, L]; weight [C, 1, K]; bias [C] or None;
    state_in [B, carry, C] / [B, C, carry] with a leading [W] axis when state_window = W,
    or None (zeros); carry = (K - 1) * dilation.  ``state_out`` may be ``state_in``."""
    lib = load()
    B, L, C, K = _conv_geometry(x, weight, channels_last)
    dt = x.dtype
    _need_cuda("x", x, dt)
    _need_cuda("weight", weight, dt)
    if bias is not None:
        _need_cuda("bias", bias, dt)
        if tuple(bias.shape) != (C,):
            raise GdnError(GDN_ERR_INVALID_ARG, f"bias must be [{C}]")
    st_shape = conv_state_shape(B, C, K, dilation, channels_last, state_window)
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None:
            _need_cuda(name, t, dt)
            if tuple(t.shape) != st_shape:
                raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be {st_shape}")
    if y is None:
        y = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        _need_cuda("y", y, dt)
    if state_out is None:
        state_out = torch.empty(st_shape, dtype=dt, device=x.device)
    shape = GdnConvShape(_DTYPE_CODE[dt], B, L, C, K, int(dilation), int(bool(channels_last)),
                         ACTIVATIONS[activation], int(state_window))
    _check(lib.gdn_causal_conv(ctypes.byref(shape), _ptr(x), _ptr(weight), _ptr(bias),
                               _ptr(state_in), _ptr(y), _ptr(state_out), _stream(stream)))
    return y, state_out


def gdn_causal_conv_slots(x, weight, pool, slots, bias=None, *, dilation: int = 1,
                          activation: str = "none", y=None, stream=None):
    """The convolution against a pool of states: row b reads and updates
    ``pool[slots[b]]`` in place.  x [B, L, C]; pool [P, carry, C]; slots int32 [B].
    Returns y [B, L, C]."""
    lib = load()
    B, L, C, K = _conv_geometry(x, weight, True)
    dt = x.dtype
    for name, t in (("x", x), ("weight", weight), ("pool", pool)):
        _need_cuda(name, t, dt)
    _need_cuda("slots", slots, torch.int32)
    carry = (K - 1) * dilation
    if pool.dim() != 3 or tuple(pool.shape[1:]) != (carry, C):
        raise GdnError(GDN_ERR_INVALID_ARG, f"pool must be [P, {carry}, {C}]")
    if tuple(slots.shape) != (B,):
        raise GdnError(GDN_ERR_INVALID_ARG, "slots must be [B]")
    if bias is not None:
        _need_cuda("bias", bias, dt)
    if y is None:
        y = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        _need_cuda("y", y, dt)
    shape = GdnConvShape(_DTYPE_CODE[dt], B, L, C, K, int(dilation), 1, ACTIVATIONS[activation], 0)
    _check(lib.gdn_causal_conv_slots(ctypes.byref(shape), _ptr(x), _ptr(weight), _ptr(bias),
                                     _ptr(pool), int(pool.shape[0]), _ptr(slots), _ptr(y),
                                     _stream(stream)))
    return y


def gdn_gated_rmsnorm(x, scale, gate, eps: float = 1e-5, activation: str = "silu", *, y=None,
                      stream=None):
    """y = x / sqrt(mean(x^2) + eps) * scale * act(gate) over rows of len(scale) values."""
    lib = load()
    dt = x.dtype
    if dt not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unsupported io dtype {dt}")
    for name, t in (("x", x), ("scale", scale), ("gate", gate)):
        _need_cuda(name, t, dt)
    width = scale.numel()
    if scale.dim() != 1 or width == 0 or x.numel() % width != 0 or gate.shape != x.shape:
        raise GdnError(GDN_ERR_INVALID_ARG, "scale must be [C] dividing x's size; gate like x")
    if y is None:
        y = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        _need_cuda("y", y, dt)
    _check(lib.gdn_gated_rmsnorm(_DTYPE_CODE[dt], x.numel() // width, width, _ptr(x), _ptr(scale),
                                 _ptr(gate), float(eps), ACTIVATIONS[activation], _ptr(y),
                                 _stream(stream)))
    return y


def gdn_decode_layer(x, conv_weight, conv_bias, conv_state_in, conv_state_out, a, b, A_log,
                     dt_bias, state, norm_scale, gate, *, h_qk: int, h_v: int, d_k: int = 128,
                     scale: float = 0.0, conv_activation: str = "silu",
                     norm_activation: str = "silu", eps: float = 1e-5, y=None, stream=None):
    """One decode token of the layer: causal conv over x [B, 1, C] (channels read as
    [q | k | v], C = 2 h_qk d_k + h_v d_v), the gated delta-rule step on state
    [B, h_v, d_k, d_v] (in place), then the gated RMS norm of o with norm_scale [d_v] and
    gate [B, 1, h_v, d_v].  conv_weight [C, 1, K]; conv_bias [C] or None; conv states
    [B, K - 1, C] (conv_state_in None = zeros; conv_state_out None = not written; the two
    may not overlap).  Returns y [B, 1, h_v, d_v]."""
    lib = load()
    dt = x.dtype
    if dt not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unsupported io dtype {dt}")
    for name, t in (("x", x), ("conv_weight", conv_weight), ("a", a), ("b", b),
                    ("norm_scale", norm_scale), ("gate", gate)):
        _need_cuda(name, t, dt)
    for name, t in (("conv_bias", conv_bias), ("conv_state_in", conv_state_in),
                    ("conv_state_out", conv_state_out)):
        if t is not None:
            _need_cuda(name, t, dt)
    _need_cuda("state", state, torch.float32)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    if x.dim() != 3 or x.shape[1] != 1:
        raise GdnError(GDN_ERR_INVALID_ARG, "x must be [B, 1, C]")
    B, C = x.shape[0], x.shape[2]
    d_v = norm_scale.numel()
    if C != 2 * h_qk * d_k + h_v * d_v or conv_weight.numel() % C != 0:
        raise GdnError(GDN_ERR_INVALID_ARG, "x's channels must be 2 h_qk d_k + h_v d_v; weight [C, 1, K]")
    K = conv_weight.numel() // C
    if y is None:
        y = torch.empty((B, 1, h_v, d_v), dtype=dt, device=x.device)
    else:
        _need_cuda("y", y, dt)
    shape = make_shape(_DTYPE_CODE[dt], B, 1, B, h_qk, h_v, d_k, d_v)
    layer = GdnLayerParams(K, ACTIVATIONS[conv_activation], ACTIVATIONS[norm_activation], float(eps))
    _check(lib.gdn_decode_layer(ctypes.byref(shape), ctypes.byref(layer), _ptr(x), _ptr(conv_weight),
                                _ptr(conv_bias), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(a),
                                _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(state), float(scale),
                                _ptr(norm_scale), _ptr(gate), _ptr(y), _stream(stream)))
    return y


def gdn_prefill_layer(x, conv_weight, conv_bias, conv_state_in, a, b, A_log, dt_bias, state_in,
                      cu_seqlens, norm_scale, gate, *, h_qk: int, h_v: int, scale: float = 0.0,
                      conv_activation: str = "silu", norm_activation: str = "silu", eps: float = 1e-5,
                      fuse: bool = False, y=None, state_out=None, conv_state_out=None, workspace=None,
                      stream=None):
    """The prefill of a layer: causal conv over x (channels [q | k | v], C = 2 h_qk 128 +
    h_v 128; [B, T, C], or [1, total, C] packed with cu_seqlens), the chunked prefill on its
    q, k, v, then the gated RMS norm of o.  conv_weight [C, 1, K] (K <= 4); conv_bias [C] or
    None; conv_state_in [N, K - 1, C] or None (zeros).  Returns (y [.., h_v, 128],
    state_out [N, h_v, 128, 128], conv_state_out [N, K - 1, C])."""
    lib = load()
    dt = x.dtype
    if dt not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, f"unsupported io dtype {dt}")
    for name, t in (("x", x), ("conv_weight", conv_weight), ("a", a), ("b", b),
                    ("norm_scale", norm_scale), ("gate", gate)):
        _need_cuda(name, t, dt)
    for name, t in (("conv_bias", conv_bias), ("conv_state_in", conv_state_in)):
        if t is not None:
            _need_cuda(name, t, dt)
    _need_cuda("A_log", A_log, torch.float32)
    _need_cuda("dt_bias", dt_bias, torch.float32)
    if x.dim() != 3:
        raise GdnError(GDN_ERR_INVALID_ARG, "x must be [B, T, C]")
    B, T, C = x.shape
    d = 128
    if C != 2 * h_qk * d + h_v * d or conv_weight.numel() % C != 0:
        raise GdnError(GDN_ERR_INVALID_ARG, "x's channels must be 2 h_qk 128 + h_v 128; weight [C, 1, K]")
    K = conv_weight.numel() // C
    if cu_seqlens is not None:
        _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
        if B != 1:
            raise GdnError(GDN_ERR_INVALID_ARG, "packed sequences need x [1, total, C]")
        n_seq = cu_seqlens.numel() - 1
        shape = make_shape(_DTYPE_CODE[dt], 1, T, n_seq, h_qk, h_v, d, d)
    else:
        n_seq = B
        shape = make_shape(_DTYPE_CODE[dt], B, T, B, h_qk, h_v, d, d)
    if state_in is not None:
        _need_cuda("state_in", state_in, torch.float32)
    if y is None:
        y = torch.empty((B, T, h_v, d), dtype=dt, device=x.device)
    if state_out is None:
        state_out = torch.empty((n_seq, h_v, d, d), dtype=torch.float32, device=x.device)
    if conv_state_out is None:
        conv_state_out = torch.empty((n_seq, max(K - 1, 0), C), dtype=dt, device=x.device)
    need = int(lib.gdn_prefill_layer_workspace_bytes(ctypes.byref(shape)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    layer = GdnLayerParams(K, ACTIVATIONS[conv_activation], ACTIVATIONS[norm_activation], float(eps))
    _check(lib.gdn_prefill_layer(ctypes.byref(shape), ctypes.byref(layer), _ptr(x), _ptr(conv_weight),
                                 _ptr(conv_bias), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(a),
                                 _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(state_in), _ptr(cu_seqlens),
                                 float(scale), _ptr(norm_scale), _ptr(gate), _ptr(y), _ptr(state_out),
                                 int(bool(fuse)), _ptr(workspace), ws_bytes, _stream(stream)))
    return y, state_out, conv_state_out


# ------------------------------------------------------------------ the state-space layer
def _bad(name: str, t, shape, dtype, device: int):
    """Say what _arg found wrong with a tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be on cuda:{device}, as the call's first tensor is")
    if t.dtype != dtype:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be contiguous")


def _arg(name: str, t, shape, dtype, device: int):
    """Address of a contiguous tensor of this shape (None: any), type and device; None passes."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype != dtype or not t.is_contiguous() or \
            (shape is not None and t.shape != shape):
        _bad(name, t, shape, dtype, device)
    return t.data_ptr()


def _rows(name: str, t, B: int, T: int, row: tuple, dtype, device: int):
    """(address, elements between token rows) of t [B, T, *row], whose token rows are contiguous in
    themselves and evenly spaced."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype != dtype or t.shape != (B, T) + row:
        _bad(name, t, (B, T) + row, dtype, device)
    stride, step = t.stride(), 1
    for n, s in zip(reversed(row), reversed(stride[2:])):
        if n > 1 and s != step:
            raise GdnError(GDN_ERR_INVALID_ARG, f"{name}'s token rows must be contiguous")
        step *= n
    if T > 1 and B > 1 and stride[0] != T * stride[1]:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name}'s token rows must be evenly spaced over the batch")
    apart = stride[1] if T > 1 else stride[0] if B > 1 else step
    if apart < step and B * T > 1:      # (0, as of an expanded tensor, would be taken for contiguous rows)
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name}'s token rows must not overlap (an expanded tensor has to be copied)")
    return t.data_ptr(), apart


@contextlib.contextmanager
def _elsewhere(device: int, stream):
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
        raise GdnError(GDN_ERR_INVALID_ARG, f"stream must be on cuda:{device}, as the call's first tensor is")
    with torch.cuda.device(device):
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            yield


_HERE = contextlib.nullcontext()


def _on(device: int, stream):
    """The context a call allocates and launches in: its tensors' device, and the stream's own
    memory pool when it names one (a workspace freed on return is then reused in its order)."""
    return _HERE if stream is None and torch.cuda.current_device() == device else _elsewhere(device, stream)


def _raw_stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


def _first(name: str, t, dims: int) -> int:
    """Device of the call's first tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != dims or t.dtype not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must have {dims} axes, in float32, bfloat16 or float16")
    if not t.is_cuda:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    return t.get_device()


def _conv_taps(conv_weight, C: int) -> int:
    if conv_weight is None:
        return 0
    if C <= 0 or not isinstance(conv_weight, torch.Tensor) or conv_weight.dim() == 0 or conv_weight.shape[0] != C or \
            conv_weight.numel() == 0:
        raise GdnError(GDN_ERR_INVALID_ARG, f"conv_weight must be [{C}, 1, K]")
    return conv_weight.numel() // C


def gdn_ssm_prefill_workspace_bytes(shape: GdnSsmShape, params: GdnSsmParams) -> int:
    return int(load().gdn_ssm_prefill_workspace_bytes(ctypes.byref(shape), ctypes.byref(params)))


def gdn_ssm_prefill_plan(shape: GdnSsmShape, params: GdnSsmParams):
    """(path, launches) of a gdn_ssm_prefill call: PATH_SIMT, PATH_TC or PATH_TC_TP (time segments)."""
    path, launches = ctypes.c_int32(), ctypes.c_int32()
    _check(load().gdn_ssm_prefill_plan(ctypes.byref(shape), ctypes.byref(params), ctypes.byref(path), ctypes.byref(launches)))
    return path.value, launches.value


_CONV_ACT = {"none": 0, "silu": 1}


def gdn_ssm_prefill(xbc, dt, A_log, *, heads: int, head_dim: int, d_state: int, groups: int = 1, D=None, dt_bias=None,
                    z=None, conv_weight=None, conv_bias=None, conv_state_in=None, conv_activation: str = "silu",
                    state_in=None, cu_seqlens=None, dt_min: float = 0.0, dt_max: float = float("inf"), y=None,
                    state_out=None, conv_state_out=None, workspace=None, stream=None):
    """The selective state-space scan over whole sequences, behind its short causal convolution.

    xbc [B, T, C], C = heads head_dim + 2 groups d_state, rows [x | B | C]; dt [B, T, heads]; z
    [B, T, heads, head_dim] or None: token rows may be slices of wider ones (contiguous in
    themselves, evenly spaced, none over another: copy an expanded tensor).  With cu_seqlens (int32 [N + 1]) B is 1 and T the packed total.
    conv_weight [C, 1, K] (K <= 4) and conv_bias [C], or None: xbc is taken as it is.
    conv_state_in [N, K - 1, C], state_in [N, heads, d_state, head_dim] fp32: zeros when None.
    A_log, dt_bias, D [heads] fp32.  Returns (y [B, T, heads, head_dim], state_out,
    conv_state_out or None)."""
    lib = _lib or load()
    dev = _first("xbc", xbc, 3)
    if conv_activation not in _CONV_ACT:
        raise GdnError(GDN_ERR_INVALID_ARG, "the convolution's activation is 'none' or 'silu'")
    io, (B, T, _) = xbc.dtype, xbc.shape
    C = heads * head_dim + 2 * groups * d_state
    K = _conv_taps(conv_weight, C)
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    f32, states, convs = torch.float32, (max(n, 0), heads, d_state, head_dim), (max(n, 0), max(K - 1, 0), C)
    px, ldx = _rows("xbc", xbc, B, T, (C,), io, dev)
    pdt, lddt = _rows("dt", dt, B, T, (heads,), io, dev)
    pz, ldz = (None, 0) if z is None else _rows("z", z, B, T, (heads, head_dim), io, dev)
    per_head, chan = (heads,), (C,)
    pcu = _arg("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, dev)
    pA, pb, pD = (_arg("A_log", A_log, per_head, f32, dev), _arg("dt_bias", dt_bias, per_head, f32, dev),
                  _arg("D", D, per_head, f32, dev))
    pw, pcb = _arg("conv_weight", conv_weight, None, io, dev), _arg("conv_bias", conv_bias, chan, io, dev)
    psi, pci = _arg("state_in", state_in, states, f32, dev), _arg("conv_state_in", conv_state_in, convs, io, dev)
    shape = GdnSsmShape(_DTYPE_CODE[io], B, T, n, heads, head_dim, groups, d_state, ldx, lddt, ldz)
    params = GdnSsmParams(K, _CONV_ACT[conv_activation], dt_min, dt_max)
    rs, rp = ctypes.byref(shape), ctypes.byref(params)
    with _on(dev, stream):
        if y is None:
            y = torch.empty((B, T, heads, head_dim), dtype=io, device=xbc.device)
        if state_out is None:
            state_out = torch.empty(states, dtype=f32, device=xbc.device)
        if conv_state_out is None and K:
            conv_state_out = torch.empty(convs, dtype=io, device=xbc.device)
        need = lib.gdn_ssm_prefill_workspace_bytes(rs, rp)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=xbc.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(lib.gdn_ssm_prefill(rs, rp, px, pdt, pz, pw, pcb, pci, _arg("conv_state_out", conv_state_out, convs, io, dev),
                                   pA, pb, pD, psi, pcu, _arg("y", y, (B, T, heads, head_dim), io, dev),
                                   _arg("state_out", state_out, states, f32, dev),
                                   None if workspace is None else _arg("workspace", workspace, None, workspace.dtype, dev),
                                   ws_bytes, _raw_stream(dev)))
    return y, state_out, conv_state_out


def gdn_ssm_decode(xbc, dt, A_log, state, *, heads: int, head_dim: int, d_state: int, groups: int = 1, D=None, dt_bias=None,
                   z=None, conv_weight=None, conv_bias=None, conv_state=None, conv_activation: str = "silu", slots=None,
                   dt_min: float = 0.0, dt_max: float = float("inf"), y=None, stream=None):
    """One token of the state-space layer per row: gdn_ssm_prefill's arguments at T = 1, with
    ``state`` [E, heads, d_state, head_dim] fp32 and ``conv_state`` [E, K - 1, C] advanced in
    place.  With slots (int32 [B], distinct) row b uses entry slots[b], else entry b (E = B).
    Returns y [B, 1, heads, head_dim]."""
    lib = _lib or load()
    dev = _first("xbc", xbc, 3)
    if conv_activation not in _CONV_ACT:
        raise GdnError(GDN_ERR_INVALID_ARG, "the convolution's activation is 'none' or 'silu'")
    io, (B, T, _) = xbc.dtype, xbc.shape
    C = heads * head_dim + 2 * groups * d_state
    K = _conv_taps(conv_weight, C)
    if K > 1 and conv_state is None:
        raise GdnError(GDN_ERR_INVALID_ARG, "conv_state is needed with conv_weight")
    E = state.shape[0] if slots is not None and isinstance(state, torch.Tensor) and state.dim() == 4 else B
    f32, per_head = torch.float32, (heads,)
    px, ldx = _rows("xbc", xbc, B, T, (C,), io, dev)
    pdt, lddt = _rows("dt", dt, B, T, (heads,), io, dev)
    pz, ldz = (None, 0) if z is None else _rows("z", z, B, T, (heads, head_dim), io, dev)
    shape = GdnSsmShape(_DTYPE_CODE[io], B, T, B, heads, head_dim, groups, d_state, ldx, lddt, ldz)
    params = GdnSsmParams(K, _CONV_ACT[conv_activation], dt_min, dt_max)
    with _on(dev, stream):
        if y is None:
            y = torch.empty((B, T, heads, head_dim), dtype=io, device=xbc.device)
        if state is None:
            raise GdnError(GDN_ERR_INVALID_ARG, "state is needed")
        _check(lib.gdn_ssm_decode(ctypes.byref(shape), ctypes.byref(params), px, pdt, pz,
                                  _arg("conv_weight", conv_weight, None, io, dev), _arg("conv_bias", conv_bias, (C,), io, dev),
                                  _arg("conv_state", conv_state, (E, K - 1, C), io, dev) if K else None,
                                  _arg("A_log", A_log, per_head, f32, dev), _arg("dt_bias", dt_bias, per_head, f32, dev),
                                  _arg("D", D, per_head, f32, dev),
                                  _arg("state", state, (E, heads, d_state, head_dim), f32, dev), E,
                                  _arg("slots", slots, (B,), torch.int32, dev),
                                  _arg("y", y, (B, T, heads, head_dim), io, dev), _raw_stream(dev)))
    return y


# ------------------------------------------------------------------ the diagonal recurrence
# The device time of a small call is a few microseconds, so what a call's sizes say is worked out once for each set of them.
@functools.lru_cache(maxsize=1024)
def _diag_shape(io, B, T, n, C, gate, weighting, has_b, keep, *strides):
    """(reference to the shape, bytes kept, workspace bytes of the forward and of the backward pass)."""
    if gate not in DIAG_GATES or weighting not in DIAG_WEIGHTINGS or keep not in DIAG_KEEPS:
        raise GdnError(GDN_ERR_INVALID_ARG, f"gate must be one of {sorted(DIAG_GATES)}, weighting of {sorted(DIAG_WEIGHTINGS)}, "
                                            "keep None, 'states' or '8bit'")
    if max(B, n, C) > 2 ** 31 - 1:          # (the shape's fields would keep their low 32 bits)
        raise GdnError(GDN_ERR_UNSUPPORTED, f"a batch of {B}, {n} sequences or {C} channels is not built")
    lib = load()
    ref = ctypes.byref(GdnDiagShape(_DTYPE_CODE[io], B, T, n, C, DIAG_GATES[gate], DIAG_WEIGHTINGS[weighting], has_b, DIAG_KEEPS[keep], *strides))
    return ref, lib.gdn_diag_kept_bytes(ref), lib.gdn_diag_prefill_workspace_bytes(ref), lib.gdn_diag_backward_workspace_bytes(ref)


def _row3(name: str, t, rows, dtype, device: int):
    """_rows for t [B, T, C]; what lies as it mostly does is seen at once."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == rows and t.get_device() == device:
        (B, T, C), (s0, s1, s2) = rows, t.stride()
        if s2 == 1 and (s1 >= C and s0 == T * s1 if T > 1 else s0 >= C):
            return t.data_ptr(), s1 if T > 1 else s0
    return _rows(name, t, rows[0], rows[1], (rows[2],), dtype, device)


def _diag_params(A_log, a_bias, b_bias, C: int, input_gate: bool, dev: int):
    if b_bias is not None and not input_gate:
        raise GdnError(GDN_ERR_INVALID_ARG, "b_bias belongs to an input gate: b is needed")
    if A_log is None:
        raise GdnError(GDN_ERR_INVALID_ARG, "A_log is needed")
    per, f32 = (C,), torch.float32
    return _arg("A_log", A_log, per, f32, dev), _arg("a_bias", a_bias, per, f32, dev), _arg("b_bias", b_bias, per, f32, dev)


def _workspace(workspace, need: int, device, dev: int):
    """(the workspace, its address, its bytes), made where it is needed and not given."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, _arg("workspace", workspace, None, workspace.dtype, dev), workspace.numel() * workspace.element_size()


def gdn_diag_kept_bytes(shape: GdnDiagShape) -> int:
    return int(load().gdn_diag_kept_bytes(ctypes.byref(shape)))


def gdn_diag_prefill_workspace_bytes(shape: GdnDiagShape) -> int:
    return int(load().gdn_diag_prefill_workspace_bytes(ctypes.byref(shape)))


def gdn_diag_backward_workspace_bytes(shape: GdnDiagShape) -> int:
    return int(load().gdn_diag_backward_workspace_bytes(ctypes.byref(shape)))


def gdn_diag_prefill(x, a, b, A_log, *, a_bias=None, b_bias=None, gate: str = "softplus", weighting: str = "norm", state_in=None,
                     cu_seqlens=None, keep=None, y=None, state_out=None, kept=None, workspace=None, stream=None):
    """The diagonal recurrence over whole sequences: h_t = alpha_t h_{t-1} + w_t sigmoid(b_t + b_bias) x_t per channel, with
    alpha_t = exp(-exp(A_log) softplus(a_t + a_bias)) (gate 'softplus') or exp(-exp(A_log) sigmoid(a_t + a_bias))
    ('sigmoid') and w_t = 1 ('plain'), 1 - alpha_t ('complement') or sqrt(1 - alpha_t^2) ('norm').

    x, a, b [B, T, C] (b None: no input gate); token rows may be slices of wider ones (contiguous in themselves, evenly
    spaced, none over another).  With cu_seqlens (int32 [N + 1]) B is 1 and T the packed total.  A_log, a_bias, b_bias
    [C] fp32; state_in [N, C] fp32 or None (zeros).  -infinity in a or b holds that gate shut.  keep: what a backward pass will need, 'states' (beside x, a and b
    themselves), '8bit' (instead of them) or None; `kept` may give the uint8 buffer.  No autograd graph is recorded, whatever the
    inputs require: gradients are gdn_diag_backward's.  Returns (y, state_out, a GdnDiagKept or None)."""
    lib = _lib or load()
    dev = _first("x", x, 3)
    io, rows, has_b, f32 = x.dtype, x.shape, b is not None, torch.float32
    B, T, C = rows
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    states = (max(n, 0), C)
    px, ldx = _row3("x", x, rows, io, dev)
    pa, lda = _row3("a", a, rows, io, dev)
    pb, ldb = _row3("b", b, rows, io, dev) if has_b else (None, 0)
    pA, pab, pbb = _diag_params(A_log, a_bias, b_bias, C, has_b, dev)
    pcu = _arg("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, dev)
    psi = _arg("state_in", state_in, states, f32, dev)
    with _on(dev, stream):
        if y is None:
            y = torch.empty(rows, dtype=io, device=x.device)
        if state_out is None:
            state_out = torch.empty(states, dtype=f32, device=x.device)
        py, ldy = _row3("y", y, rows, io, dev)
        ref, bytes_, need, _ = _diag_shape(io, B, T, n, C, gate, weighting, has_b, keep, ldx, lda, ldb, ldy)
        if keep is not None and kept is None:
            kept = torch.empty(bytes_, dtype=torch.uint8, device=x.device)
        workspace, pw, ws_bytes = _workspace(workspace, need, x.device, dev)
        _check(lib.gdn_diag_prefill(ref, px, pa, pb, pA, pab, pbb, psi, pcu, py, _arg("state_out", state_out, states, f32, dev),
                                    _arg("kept", kept, None, torch.uint8, dev), 0 if kept is None else kept.numel(), pw, ws_bytes,
                                    _raw_stream(dev)))
    return y, state_out, None if keep is None else GdnDiagKept(kept, io, B, T, n, C, gate, weighting, has_b, keep)


def gdn_diag_backward(dy, kept: GdnDiagKept, A_log, *, x=None, a=None, b=None, a_bias=None, b_bias=None, state_in=None,
                      cu_seqlens=None, dstate_out=None, dx=None, da=None, db=None, workspace=None, stream=None):
    """The gradients of sum(y dy) + sum(state_out dstate_out) of a gdn_diag_prefill call, from what it kept.

    dy [B, T, C]; dstate_out [N, C] fp32 or None (zeros); A_log, the biases, state_in and cu_seqlens as the forward
    call had them, and x, a, b too unless it kept '8bit' (they are then not read, and the gradients are those at the
    values that the codes hold).  dx, da, db may give their rows, as slices of a wider one too.  Returns (dx, da, db,
    dA_log, da_bias, db_bias, dstate_in), None for what the forward call did not have."""
    lib = _lib or load()
    if not isinstance(kept, GdnDiagKept):
        raise GdnError(GDN_ERR_INVALID_ARG, "kept must be what gdn_diag_prefill kept")
    dev = _first("dy", dy, 3)
    data, io, B, T, n, C, gate, weighting, has_b, keep = kept
    f32, states, rows = torch.float32, (max(n, 0), C), (B, T, C)
    pdy, lddy = _row3("dy", dy, rows, io, dev)
    pA, pab, pbb = _diag_params(A_log, a_bias, b_bias, C, has_b, dev)
    pcu = _arg("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, dev)
    if cu_seqlens is None and n != B:
        raise GdnError(GDN_ERR_INVALID_ARG, "cu_seqlens is needed: the forward call was packed")
    psi, pdo = _arg("state_in", state_in, states, f32, dev), _arg("dstate_out", dstate_out, states, f32, dev)
    pk = _arg("kept", data, None, torch.uint8, dev)
    px = pa = pb = None
    ldx = lda = ldb = 0
    if keep == "states":
        px, ldx = _row3("x", x, rows, io, dev)
        pa, lda = _row3("a", a, rows, io, dev)
        if has_b:
            pb, ldb = _row3("b", b, rows, io, dev)
    with _on(dev, stream):
        new = lambda shape, dtype=f32: torch.empty(shape, dtype=dtype, device=dy.device)  # noqa: E731
        dx, da = new(rows, io) if dx is None else dx, new(rows, io) if da is None else da
        db = None if not has_b else new(rows, io) if db is None else db
        pdx, lddx = _row3("dx", dx, rows, io, dev)
        pda, ldda = _row3("da", da, rows, io, dev)
        pdb, lddb = _row3("db", db, rows, io, dev) if has_b else (None, 0)
        dA_log, da_bias, db_bias = new((C,)), None if a_bias is None else new((C,)), None if b_bias is None else new((C,))
        dstate_in = None if state_in is None else new(states)
        ref, _, _, need = _diag_shape(io, B, T, n, C, gate, weighting, has_b, keep, ldx, lda, ldb, lddy, lddx, ldda, lddb)
        workspace, pw, ws_bytes = _workspace(workspace, need, dy.device, dev)
        _check(lib.gdn_diag_backward(ref, px, pa, pb, pA, pab, pbb, psi, pcu, pk, data.numel(), pdy, pdo, pdx, pda, pdb,
                                     *(None if t is None else t.data_ptr() for t in (dA_log, da_bias, db_bias, dstate_in)), pw,
                                     ws_bytes, _raw_stream(dev)))
    return dx, da, db, dA_log, da_bias, db_bias, dstate_in


def gdn_diag_decode(x, a, b, A_log, state, *, a_bias=None, b_bias=None, gate: str = "softplus", weighting: str = "norm",
                    slots=None, y=None, stream=None):
    """One token of the diagonal recurrence per row: gdn_diag_prefill's arguments at T = 1, with ``state`` [E, C] fp32
    advanced in place.  With slots (int32 [B], distinct) row b uses entry slots[b], else entry b (E = B).  Returns y
    [B, 1, C]."""
    lib = _lib or load()
    dev = _first("x", x, 3)
    io, rows, has_b = x.dtype, x.shape, b is not None
    B, T, C = rows
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise GdnError(GDN_ERR_INVALID_ARG, f"state must be [E, {C}]")
    E = B if slots is None else state.shape[0]
    px, ldx = _row3("x", x, rows, io, dev)
    pa, lda = _row3("a", a, rows, io, dev)
    pb, ldb = _row3("b", b, rows, io, dev) if has_b else (None, 0)
    pA, pab, pbb = _diag_params(A_log, a_bias, b_bias, C, has_b, dev)
    ps, pslots = _arg("state", state, (E, C), torch.float32, dev), _arg("slots", slots, (B,), torch.int32, dev)
    with _on(dev, stream):
        if y is None:
            y = torch.empty(rows, dtype=io, device=x.device)
        py, ldy = _row3("y", y, rows, io, dev)
        ref = _diag_shape(io, B, T, B, C, gate, weighting, has_b, None, ldx, lda, ldb, ldy)[0]
        _check(lib.gdn_diag_decode(ref, px, pa, pb, pA, pab, pbb, ps, E, pslots, py, _raw_stream(dev)))
    return y


def gdn_checkpoint_pack(x, *, codes=None, steps=None, stream=None):
    """x [B, T, C] (token rows may be slices of wider ones) in 8 bits: (codes int8 [B, T, C], steps uint8 [B, T,
    ceil(C / 64)]).  64 channels of a row share the step 2^(s - 133), the least at which they round within 127; one
    with an infinity or a NaN among them is read back as NaN."""
    lib = _lib or load()
    dev = _first("x", x, 3)
    B, T, C = x.shape
    px, ldx = _row3("x", x, x.shape, x.dtype, dev)
    blocks = (B, T, -(-C // CHECKPOINT_BLOCK))
    with _on(dev, stream):
        if codes is None:
            codes = torch.empty((B, T, C), dtype=torch.int8, device=x.device)
        if steps is None:
            steps = torch.empty(blocks, dtype=torch.uint8, device=x.device)
        _check(lib.gdn_checkpoint_pack(_DTYPE_CODE[x.dtype], B * T, C, px, ldx, _arg("codes", codes, (B, T, C), torch.int8, dev),
                                       _arg("steps", steps, blocks, torch.uint8, dev), _raw_stream(dev)))
    return codes, steps


def gdn_checkpoint_unpack(codes, steps, dtype=torch.bfloat16, *, y=None, stream=None):
    """The rows that gdn_checkpoint_pack packed, [B, T, C] in dtype: exact in bfloat16 and float32, held to the largest
    finite value in float16."""
    lib = _lib or load()
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3 or not codes.is_cuda or dtype not in _DTYPE_CODE:
        raise GdnError(GDN_ERR_INVALID_ARG, "codes must be a CUDA tensor of 3 axes, dtype float32, bfloat16 or float16")
    dev, (B, T, C) = codes.get_device(), codes.shape
    pc = _arg("codes", codes, None, torch.int8, dev)
    ps = _arg("steps", steps, (B, T, -(-C // CHECKPOINT_BLOCK)), torch.uint8, dev)
    with _on(dev, stream):
        if y is None:
            y = torch.empty((B, T, C), dtype=dtype, device=codes.device)
        py, ldy = _row3("y", y, codes.shape, dtype, dev)
        _check(lib.gdn_checkpoint_unpack(_DTYPE_CODE[dtype], B * T, C, pc, ps, py, ldy, _raw_stream(dev)))
    return y


# ------------------------------------------------------------------ rotary positions
def gdn_rotary_frequencies(rot_dim: int, base: float = 10000.0, kind: str = "plain", *, factor: float = 1.0,
                           trained_length: float = 0.0, low: float = 1.0, high: float = 32.0, device=None):
    """(inv_freq [rot_dim / 2] fp32, scale) for gdn_rotary: 'plain'; 'linear' (positions / factor:
    position interpolation); 'base' (the base grown by factor: NTK-aware scaling); 'bands' (YaRN) and
    'wavelength' (frequencies that turn less than `low` times over trained_length divided by factor,
    those above `high` times kept, a ramp between, over the indices or over the turns)."""
    if kind not in ROTARY_KINDS:
        raise GdnError(GDN_ERR_INVALID_ARG, f"kind must be one of {sorted(ROTARY_KINDS)}")
    inv_freq = torch.empty(max(rot_dim, 0) // 2, dtype=torch.float32)
    scale = ctypes.c_float()
    scaling = GdnRotaryScaling(ROTARY_KINDS[kind], base, factor, trained_length, low, high)
    _check(load().gdn_rotary_frequencies(ctypes.byref(scaling), rot_dim, ctypes.c_void_p(inv_freq.data_ptr()),
                                         ctypes.byref(scale)))
    return inv_freq.to(device) if device is not None else inv_freq, scale.value


def _heads(name: str, t, shape, dtype, device: int):
    """(address, row stride, head stride) of t [B, T, H, D], whose rows are evenly spaced."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype != dtype or t.shape != shape:
        _bad(name, t, shape, dtype, device)
    B, T, H, D = shape
    s0, s1, s2, s3 = t.stride()
    if D > 1 and s3 != 1:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name}'s heads must be contiguous")
    head = s2 if H > 1 else D
    if T > 1 and B > 1 and s0 != T * s1:
        raise GdnError(GDN_ERR_INVALID_ARG, f"{name}'s token rows must be evenly spaced over the batch")
    return t.data_ptr(), s1 if T > 1 else s0 if B > 1 else max(H * head, D), head


def gdn_rotary(q, k, inv_freq, *, positions=None, cu_seqlens=None, rot_offset: int = 0, interleaved: bool = False,
               inverse: bool = False, scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions on q [B, T, Hq, D] and k [B, T, Hk, D] (or None) in one launch.

    inv_freq [rot_dim / 2] fp32 turns dimensions [rot_offset, rot_offset + rot_dim) in pairs
    (2i, 2i + 1) when interleaved, else (i, i + rot_dim / 2); the rest is copied.  positions
    int32 [B, T], or None: a token's place in its sequence (cu_seqlens int32 [N + 1] when packed).
    Heads may be slices of wider rows.  q_out / k_out may be q / k.  Returns (q_out, k_out)."""
    lib = _lib or load()
    dev = _first("q", q, 4)
    io, (B, T, hq, D) = q.dtype, q.shape
    pq, qr, qh = _heads("q", q, q.shape, io, dev)
    pk, kr, kh, hk = None, 0, 0, 0
    if k is not None:
        hk = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
        pk, kr, kh = _heads("k", k, (B, T, hk, D), io, dev)
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise GdnError(GDN_ERR_INVALID_ARG, "inv_freq must be [rot_dim / 2]")
    pf = _arg("inv_freq", inv_freq, None, torch.float32, dev)
    pp = _arg("positions", positions, (B, T), torch.int32, dev)
    pc = _arg("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, dev)
    with _on(dev, stream):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=io, device=q.device)
        if k_out is None and k is not None:
            k_out = torch.empty(k.shape, dtype=io, device=q.device)
        pqo, qor, qoh = _heads("q_out", q_out, q.shape, io, dev)
        pko, kor, koh = (None, 0, 0) if k is None else _heads("k_out", k_out, k.shape, io, dev)
        shape = GdnRotaryShape(_DTYPE_CODE[io], B, T, n, hq, hk, D, 2 * inv_freq.shape[0], rot_offset, bool(interleaved),
                               bool(inverse), scale, qr, qh, kr, kh, qor, qoh, kor, koh)
        _check(lib.gdn_rotary(ctypes.byref(shape), pq, pk, pf, pp, pc, pqo, pko, _raw_stream(dev)))
    return q_out, k_out
