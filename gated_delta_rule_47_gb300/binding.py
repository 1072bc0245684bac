"""Thin ctypes binding of libgdn.so (argument marshalling only).

Every function here checks that its tensors are CUDA, contiguous and of the
expected dtype and shape, allocates the outputs with torch, and calls the C
entry point of the same name with raw device pointers and the current CUDA
stream.  All computation happens in the library's kernels; there is no
fallback: if ``libgdn.so`` is missing or fails to load, ``load()`` raises.

The layer operators, whose smallest calls are bound by the host, go through
a native module (``build.front_path``) first, which does the same for calls in
which all is well and declines the others.  It is loaded by the first call of
one of them; the other operators need ``libgdn.so`` alone.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import importlib.machinery
import importlib.util
import math
import os
import threading

import torch

from .build import front_path

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libgdn.so")
FRONT_PATH = front_path(torch.__version__)

GDN_F32, GDN_BF16 = 0, 1
GDN_QK_L2NORM = 1
GDN_PATH_SIMT = 2
GDN_CAM_REVERSE = 4
GDN_G_PER_HEAD = 8
GDN_DT_SOFTPLUS = 16
GDN_SILU = 32
GDN_GATE_FIRST = 64
GDN_GATE_SIGMOID = 128
GDN_W_SHARED = 256
STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_MISALIGNED",
          4: "GDN_ERR_WORKSPACE", 5: "GDN_ERR_CUDA", 6: "GDN_ERR_TIMEOUT"}

EXPORTS = ("gdn_status_string", "gdn_version", "gdn_chunk_fwd_workspace_bytes", "gdn_chunk_fwd",
           "deltaproduct_chunk_fwd", "cam_prep_fwd", "gdn_get_device_error", "gdn_set_wait_limit", "gdn_launch_count",
           "gdn_set_cluster_shape", "gdn_chunk_fwd_noalloc", "cam_scan_fwd_workspace_bytes", "cam_scan_fwd",
           "masked_deltaproduct_chunk_fwd", "masked_deltaproduct_chunk_fwd_workspace_bytes",
           "cam_prep_scan_fwd_workspace_bytes", "cam_prep_scan_fwd",
           "cam_prep_bwd", "cam_scan_bwd_workspace_bytes", "cam_scan_bwd", "gdn_chunk_bwd_workspace_bytes",
           "gdn_chunk_bwd", "deltaproduct_chunk_bwd", "masked_deltaproduct_chunk_bwd_workspace_bytes",
           "masked_deltaproduct_chunk_bwd",
           "linattn_chunk_fwd_workspace_bytes", "linattn_chunk_fwd", "linattn_chunk_bwd_workspace_bytes",
           "linattn_chunk_bwd", "linattn_step", "gdn_step", "rms_norm_fwd", "rms_norm_bwd_workspace_bytes",
           "rms_norm_bwd", "state_pool_copy", "state_pool_fork_workspace_bytes", "state_pool_fork", "state_pool_free",
           "state_pool_compact_workspace_bytes", "state_pool_compact",
           "causal_conv_fwd", "causal_conv_bwd_workspace_bytes", "causal_conv_bwd", "causal_conv_step",
           "ssm_scan_fwd_workspace_bytes", "ssm_scan_fwd", "ssm_scan_bwd_workspace_bytes", "ssm_scan_bwd", "ssm_step",
           "gated_norm_fwd", "gated_norm_bwd_workspace_bytes", "gated_norm_bwd", "block_norm_fwd",
           "block_norm_bwd_workspace_bytes", "block_norm_bwd")

_lock = threading.Lock()
_lib = None
_front = None


class GdnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libgdn.so (built by ``gated_delta_rule_47_gb300.build``) and declare
    the signatures of its entry points."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libgdn.so not found at {p}; build it with "
                               "`python -m gated_delta_rule_47_gb300.build`")
        lib = ctypes.CDLL(p)
        vp, i, u, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_float, ctypes.c_size_t
        lib.gdn_status_string.argtypes = [i]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_version.restype = i
        lib.gdn_chunk_fwd_workspace_bytes.argtypes = [i] * 8
        lib.gdn_chunk_fwd_workspace_bytes.restype = sz
        lib.gdn_chunk_fwd.argtypes = [vp] * 8 + [i] * 6 + [f, u, i, vp, sz, vp]
        lib.gdn_chunk_fwd.restype = i
        lib.gdn_chunk_fwd_noalloc.argtypes = [vp] * 8 + [i] * 6 + [f, u, i, vp]
        lib.gdn_chunk_fwd_noalloc.restype = i
        lib.deltaproduct_chunk_fwd.argtypes = [vp] * 8 + [i] * 7 + [f, u, i, vp, sz, vp]
        lib.deltaproduct_chunk_fwd.restype = i
        lib.masked_deltaproduct_chunk_fwd.argtypes = [vp] * 9 + [i] * 7 + [f, u, i, vp, sz, vp]
        lib.masked_deltaproduct_chunk_fwd_workspace_bytes.argtypes = [i] * 7
        lib.masked_deltaproduct_chunk_fwd_workspace_bytes.restype = sz
        lib.masked_deltaproduct_chunk_fwd.restype = i
        lib.cam_prep_scan_fwd_workspace_bytes.argtypes = [i] * 6
        lib.cam_prep_scan_fwd_workspace_bytes.restype = sz
        lib.cam_prep_scan_fwd.argtypes = [vp] * 7 + [f] + [vp] * 5 + [i] * 5 + [f, f, f, u, i, vp, sz, vp]
        lib.cam_prep_scan_fwd.restype = i
        lib.cam_scan_bwd_workspace_bytes.argtypes = [i] * 7
        lib.cam_scan_bwd_workspace_bytes.restype = sz
        lib.cam_scan_bwd.argtypes = [vp] * 14 + [i] * 6 + [f, u, i, vp, sz, vp]
        lib.cam_scan_bwd.restype = i
        lib.gdn_chunk_bwd_workspace_bytes.argtypes = [i] * 7
        lib.gdn_chunk_bwd_workspace_bytes.restype = sz
        lib.gdn_chunk_bwd.argtypes = [vp] * 14 + [i] * 5 + [f, u, i, vp, sz, vp]
        lib.gdn_chunk_bwd.restype = i
        lib.deltaproduct_chunk_bwd.argtypes = [vp] * 14 + [i] * 6 + [f, u, i, vp, sz, vp]
        lib.deltaproduct_chunk_bwd.restype = i
        lib.masked_deltaproduct_chunk_bwd_workspace_bytes.argtypes = [i] * 7
        lib.masked_deltaproduct_chunk_bwd_workspace_bytes.restype = sz
        lib.masked_deltaproduct_chunk_bwd.argtypes = [vp] * 15 + [i] * 6 + [f, u, i, vp, sz, vp]
        lib.masked_deltaproduct_chunk_bwd.restype = i
        lib.cam_prep_bwd.argtypes = [vp] * 8 + [f] + [vp] * 8 + [i] * 4 + [f, f, i, vp]
        lib.cam_prep_bwd.restype = i
        lib.cam_scan_fwd_workspace_bytes.argtypes = [i] * 7
        lib.cam_scan_fwd_workspace_bytes.restype = sz
        lib.cam_scan_fwd.argtypes = [vp] * 8 + [i] * 6 + [f, u, i, vp, sz, vp]
        lib.cam_scan_fwd.restype = i
        lib.cam_prep_fwd.argtypes = [vp] * 9 + [f] + [vp] * 5 + [i] * 4 + [f, f, i, vp]
        lib.cam_prep_fwd.restype = i
        ll = ctypes.c_longlong
        for name in ("linattn_chunk_fwd_workspace_bytes", "linattn_chunk_bwd_workspace_bytes"):
            getattr(lib, name).argtypes = [i] * 8 + [u, i]
            getattr(lib, name).restype = sz
        lib.linattn_chunk_fwd.argtypes = [vp] * 9 + [i] * 7 + [f, u, i, vp, sz, vp]
        lib.linattn_chunk_bwd.argtypes = [vp] * 14 + [i] * 7 + [f, u, i, vp, sz, vp]
        lib.linattn_step.argtypes = [vp] * 8 + [i] * 6 + [f, u, i, vp]
        lib.gdn_step.argtypes = [vp] * 9 + [i] * 6 + [f, u, i, vp]
        lib.rms_norm_fwd.argtypes = [vp] * 6 + [ll, i, i, f, i, i, vp]
        lib.rms_norm_bwd_workspace_bytes.argtypes = [ll, i]
        lib.rms_norm_bwd.argtypes = [vp] * 6 + [ll, i, f, i, vp, sz, vp]
        lib.state_pool_copy.argtypes = [vp, i, i, ll, vp, vp, i, vp]
        lib.state_pool_fork_workspace_bytes.argtypes = [i, i]
        lib.state_pool_fork.argtypes = [vp, i, i, ll, vp, vp, vp, i, vp, sz, vp]
        lib.state_pool_free.argtypes = [vp, i, vp, i, vp]
        lib.state_pool_compact_workspace_bytes.argtypes = [i]
        lib.state_pool_compact.argtypes = [vp, i, i, ll, vp, vp, vp, vp, sz, vp]
        lib.causal_conv_fwd.argtypes = [vp] * 8 + [i] * 5 + [u, i, vp]
        lib.causal_conv_bwd_workspace_bytes.argtypes = [i] * 4
        lib.causal_conv_bwd.argtypes = [vp] * 12 + [i] * 5 + [u, i, vp, sz, vp]
        lib.causal_conv_step.argtypes = [vp] * 7 + [ll] + [i] * 4 + [u, i, vp]
        lib.ssm_scan_fwd_workspace_bytes.argtypes = [i] * 5
        lib.ssm_scan_fwd.argtypes = [vp] * 13 + [i] * 5 + [u, i, vp, sz, vp]
        lib.ssm_scan_bwd_workspace_bytes.argtypes = [i] * 5
        lib.ssm_scan_bwd.argtypes = [vp] * 22 + [i] * 5 + [u, i, vp, sz, vp]
        lib.ssm_step.argtypes = [vp] * 13 + [i] * 4 + [u, i, vp]
        lib.gated_norm_fwd.argtypes = [vp] * 5 + [i] * 4 + [f, u, i, vp]
        lib.gated_norm_bwd_workspace_bytes.argtypes = [i] * 4 + [u]
        lib.gated_norm_bwd.argtypes = [vp] * 8 + [i] * 4 + [f, u, i, vp, sz, vp]
        lib.block_norm_fwd.argtypes = [vp] * 7 + [ll, i, i, f, i, vp]
        lib.block_norm_bwd_workspace_bytes.argtypes = [ll, i, i]
        lib.block_norm_bwd.argtypes = [vp] * 12 + [ll, i, i, f, i, vp, sz, vp]
        for name in ("causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "ssm_scan_fwd", "ssm_scan_bwd", "ssm_step",
                     "gated_norm_fwd", "gated_norm_bwd", "block_norm_fwd", "block_norm_bwd"):
            getattr(lib, name).restype = i
        for name in ("rms_norm_bwd_workspace_bytes", "state_pool_fork_workspace_bytes",
                     "state_pool_compact_workspace_bytes", "causal_conv_bwd_workspace_bytes",
                     "ssm_scan_fwd_workspace_bytes", "ssm_scan_bwd_workspace_bytes", "gated_norm_bwd_workspace_bytes",
                     "block_norm_bwd_workspace_bytes"):
            getattr(lib, name).restype = sz
        for name in ("linattn_chunk_fwd", "linattn_chunk_bwd", "linattn_step", "gdn_step", "rms_norm_fwd",
                     "rms_norm_bwd", "state_pool_copy", "state_pool_fork", "state_pool_free", "state_pool_compact"):
            getattr(lib, name).restype = i
        lib.gdn_get_device_error.argtypes = [vp]
        lib.gdn_get_device_error.restype = i
        lib.gdn_set_wait_limit.argtypes = [ctypes.c_ulonglong]
        lib.gdn_set_wait_limit.restype = i
        lib.gdn_set_cluster_shape.argtypes = [i, i]
        lib.gdn_set_cluster_shape.restype = i
        lib.gdn_launch_count.restype = ctypes.c_ulonglong
        if path is None:
            _lib = lib
        return lib


def _load_front(lib):
    if not os.path.exists(FRONT_PATH):
        raise RuntimeError(f"the layer operators' module for this torch and Python is not at {FRONT_PATH}; build it with "
                           "`python -m gated_delta_rule_47_gb300.build`")
    loader = importlib.machinery.ExtensionFileLoader("_front", FRONT_PATH)
    front = importlib.util.module_from_spec(importlib.util.spec_from_loader("_front", loader))
    loader.exec_module(front)
    names = ("linattn_chunk_fwd_workspace_bytes", "linattn_chunk_fwd", "linattn_chunk_bwd_workspace_bytes",
             "linattn_chunk_bwd", "linattn_step", "gdn_step", "rms_norm_fwd", "rms_norm_bwd_workspace_bytes",
             "rms_norm_bwd", "state_pool_fork_workspace_bytes", "state_pool_fork",
             "state_pool_compact_workspace_bytes", "state_pool_compact", "causal_conv_fwd",
             "causal_conv_bwd_workspace_bytes", "causal_conv_bwd", "causal_conv_step", "ssm_scan_fwd_workspace_bytes",
             "ssm_scan_fwd", "ssm_scan_bwd_workspace_bytes", "ssm_scan_bwd", "ssm_step", "gated_norm_fwd",
             "gated_norm_bwd_workspace_bytes", "gated_norm_bwd", "block_norm_fwd", "block_norm_bwd_workspace_bytes",
             "block_norm_bwd")
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent without CUDA, where nothing asks for it
    front.init(tuple(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in names), stream, _raise)
    return front


def _quick():
    """The front, loaded."""
    global _front
    lib = load()
    with _lock:
        if _front is None:
            _front = _load_front(lib)
    return _front


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _check(t, name, shape, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _raise(fn, st):
    if st != 0:
        raise GdnError(fn, st)


def workspace_bytes(B, H, T, Dk, Dv, chunk=64, r=1, dtype=torch.bfloat16):
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    n = load().gdn_chunk_fwd_workspace_bytes(B, H, T, r, Dk, Dv, chunk, code)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("sizes rejected by gdn_chunk_fwd_workspace_bytes")
    return int(n)


def _scan(fn_name, q, k, v, beta, g, r, initial_state, output_final_state, chunk, scale, l2norm,
          o, workspace, stream, simt=False):
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    dt = q.dtype
    code = _dtype_code(q)
    sub = () if r is None else (r,)
    _check(q, "q", (B, H, T, Dk), dt)
    _check(k, "k", (B, H, T, *sub, Dk), dt)
    _check(v, "v", (B, H, T, *sub, Dv), dt)
    _check(beta, "beta", (B, H, T, *sub), dt)
    _check(g, "g", (B, H, T), torch.float32)
    if initial_state is not None:
        _check(initial_state, "initial_state", (B, H, Dk, Dv), torch.float32)
    if o is None:
        o = torch.empty(B, H, T, Dv, dtype=dt, device=q.device)
    _check(o, "o", (B, H, T, Dv), dt)
    sf = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_final_state else None
    need = workspace_bytes(B, H, T, Dk, Dv, chunk, 1 if r is None else r, dt)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lib = load()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0)
    common = [_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(initial_state), _ptr(o), _ptr(sf)]
    if r is None:
        st = lib.gdn_chunk_fwd(*common, B, H, T, Dk, Dv, chunk, float(scale), flags, code,
                               _ptr(workspace), ws_bytes, _stream(stream))
    else:
        st = lib.deltaproduct_chunk_fwd(*common, B, H, T, r, Dk, Dv, chunk, float(scale), flags, code,
                                        _ptr(workspace), ws_bytes, _stream(stream))
    _raise(fn_name, st)
    return o, sf


def gdn_chunk_fwd(q, k, v, beta, g, initial_state=None, output_final_state=False, chunk=64,
                  scale=1.0, l2norm=False, o=None, workspace=None, stream=None, simt=False):
    """Chunkwise GDN forward.  q,k [B,H,T,Dk]; v [B,H,T,Dv]; beta [B,H,T] (all
    bf16 or all fp32); g [B,H,T] fp32.  Returns (o, final_state or None).
    simt=True takes the CUDA-core path even where the tensor-core one applies."""
    return _scan("gdn_chunk_fwd", q, k, v, beta, g, None, initial_state, output_final_state, chunk,
                 scale, l2norm, o, workspace, stream, simt)


def gdn_chunk_fwd_noalloc(q, k, v, beta, g, initial_state=None, output_final_state=False, chunk=64,
                          scale=1.0, l2norm=False, o=None, stream=None):
    """gdn_chunk_fwd through the allocation-free entry point: the library uses
    its own fixed scratch array instead of a workspace (B*H <= 64 heads where
    the tensor-core path needs one).  Calls must not overlap on the GPU."""
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, T, Dk), dt)
    _check(k, "k", (B, H, T, Dk), dt)
    _check(v, "v", (B, H, T, Dv), dt)
    _check(beta, "beta", (B, H, T), dt)
    _check(g, "g", (B, H, T), torch.float32)
    if initial_state is not None:
        _check(initial_state, "initial_state", (B, H, Dk, Dv), torch.float32)
    if o is None:
        o = torch.empty(B, H, T, Dv, dtype=dt, device=q.device)
    _check(o, "o", (B, H, T, Dv), dt)
    sf = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_final_state else None
    flags = GDN_QK_L2NORM if l2norm else 0
    st = load().gdn_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(initial_state),
                                      _ptr(o), _ptr(sf), B, H, T, Dk, Dv, chunk, float(scale), flags, code,
                                      _stream(stream))
    _raise("gdn_chunk_fwd_noalloc", st)
    return o, sf


def deltaproduct_chunk_fwd(q, k, v, beta, g, initial_state=None, output_final_state=False, chunk=64,
                           scale=1.0, l2norm=False, o=None, workspace=None, stream=None, simt=False):
    """DeltaProduct forward.  q [B,H,T,Dk]; k [B,H,T,r,Dk]; v [B,H,T,r,Dv];
    beta [B,H,T,r]; g [B,H,T] fp32.  chunk counts expanded rows."""
    r = k.shape[3]
    return _scan("deltaproduct_chunk_fwd", q, k, v, beta, g, r, initial_state, output_final_state,
                 chunk, scale, l2norm, o, workspace, stream, simt)


def masked_deltaproduct_workspace_bytes(B, H, T, r, Dk, Dv, dtype=torch.bfloat16):
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(load().masked_deltaproduct_chunk_fwd_workspace_bytes(B, H, T, r, Dk, Dv, code))


def masked_deltaproduct_chunk_fwd(q, k, v, beta, g, mask, initial_state=None, output_final_state=False,
                                  chunk=64, scale=1.0, l2norm=False, o=None, workspace=None, stream=None,
                                  simt=False):
    """Block-masked DeltaProduct forward.  q, k [B,H,T,Dk]; v [B,H,T,Dv]; beta
    [B,H,T] (all bf16 or all fp32); g [B,H,T] fp32; mask [r,r] fp32 (CUDA).
    chunk counts sub-rows (tokens x r).  simt keeps the state chain on the
    CUDA cores where the tensor-core chain would run."""
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    r = mask.shape[0]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, T, Dk), dt)
    _check(k, "k", (B, H, T, Dk), dt)
    _check(v, "v", (B, H, T, Dv), dt)
    _check(beta, "beta", (B, H, T), dt)
    _check(g, "g", (B, H, T), torch.float32)
    _check(mask, "mask", (r, r), torch.float32)
    if initial_state is not None:
        _check(initial_state, "initial_state", (B, H, Dk, Dv), torch.float32)
    if o is None:
        o = torch.empty(B, H, T, Dv, dtype=dt, device=q.device)
    _check(o, "o", (B, H, T, Dv), dt)
    sf = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_final_state else None
    lib = load()
    if workspace is None:
        need = lib.masked_deltaproduct_chunk_fwd_workspace_bytes(B, H, T, r, Dk, Dv, code)
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0)
    st = lib.masked_deltaproduct_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(mask),
                                           _ptr(initial_state), _ptr(o), _ptr(sf), B, H, T, r, Dk, Dv, chunk,
                                           float(scale), flags,
                                           code, _ptr(workspace),
                                           ws_bytes, _stream(stream))
    _raise("masked_deltaproduct_chunk_fwd", st)
    return o, sf


def cam_scan_workspace_bytes(B, H, F, S, Dk, Dv, dtype=torch.bfloat16):
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    n = load().cam_scan_fwd_workspace_bytes(B, H, F, S, Dk, Dv, code)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("sizes rejected by cam_scan_fwd_workspace_bytes")
    return int(n)


def cam_scan_fwd(q, k, v, beta, decay, initial_state=None, output_final_state=False, scale=1.0,
                 reverse=False, l2norm=False, o=None, workspace=None, stream=None, simt=False):
    """Frame-level camera scan.  q, k [B,H,N,Dk]; v [B,H,N,Dv]; beta [B,H,N]
    (all bf16 or all fp32); decay [B,H,F] fp32 factors, N = F * S.  Returns
    (o, final_state or None); reverse=True is the anti-causal mode."""
    B, H, N, Dk = q.shape
    Dv = v.shape[-1]
    F = decay.shape[-1]
    if F <= 0 or N % F != 0:
        raise ValueError(f"{N} tokens do not split into {F} frames")
    S = N // F
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, N, Dk), dt)
    _check(k, "k", (B, H, N, Dk), dt)
    _check(v, "v", (B, H, N, Dv), dt)
    _check(beta, "beta", (B, H, N), dt)
    _check(decay, "decay", (B, H, F), torch.float32)
    if initial_state is not None:
        _check(initial_state, "initial_state", (B, H, Dk, Dv), torch.float32)
    if o is None:
        o = torch.empty(B, H, N, Dv, dtype=dt, device=q.device)
    _check(o, "o", (B, H, N, Dv), dt)
    sf = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_final_state else None
    need = cam_scan_workspace_bytes(B, H, F, S, Dk, Dv, dt)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0) | (GDN_CAM_REVERSE if reverse else 0)
    st = load().cam_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(decay), _ptr(initial_state), _ptr(o),
                             _ptr(sf), B, H, F, S, Dk, Dv, float(scale), flags, code, _ptr(workspace), ws_bytes,
                             _stream(stream))
    _raise("cam_scan_fwd", st)
    return o, sf


def cam_prep_scan_workspace_bytes(B, N, H, D, F, dtype=torch.bfloat16):
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    n = load().cam_prep_scan_fwd_workspace_bytes(B, N, H, D, F, code)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("sizes rejected by cam_prep_scan_fwd_workspace_bytes")
    return int(n)


def cam_prep_scan_fwd(q_raw, k_raw, v_raw, proj_q, proj_kv, beta, decay, q_norm_w=None, k_norm_w=None,
                      rope_base=10000.0, initial_state=None, output_final_state=False, k_scale=0.5, eps=1e-6,
                      scale=1.0, reverse=False, l2norm=True, o=None, workspace=None, stream=None):
    """Camera prep fused into the frame scan: raw q, k, v [B,N,H,D] bf16 ->
    o [B,H,N,D] = cam_scan_fwd(cam_prep_fwd(...)).  beta [B,H,N] bf16, decay
    [B,H,F] fp32 factors; rotation angles n * rope_base^(-2i/(D/2))."""
    B, N, H, D = q_raw.shape
    F = decay.shape[-1]
    if F <= 0 or N % F != 0:
        raise ValueError(f"{N} tokens do not split into {F} frames")
    dt = q_raw.dtype
    code = _dtype_code(q_raw)
    for name, t in (("q_raw", q_raw), ("k_raw", k_raw), ("v_raw", v_raw)):
        _check(t, name, (B, N, H, D), dt)
    _check(proj_q, "proj_q", (B, N, 4, 4), torch.float32)
    _check(proj_kv, "proj_kv", (B, N, 4, 4), torch.float32)
    _check(beta, "beta", (B, H, N), dt)
    _check(decay, "decay", (B, H, F), torch.float32)
    for name, t in (("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)):
        if t is not None:
            _check(t, name, (H * D,), torch.float32)
    if initial_state is not None:
        _check(initial_state, "initial_state", (B, H, D, D), torch.float32)
    if o is None:
        o = torch.empty(B, H, N, D, dtype=dt, device=q_raw.device)
    _check(o, "o", (B, H, N, D), dt)
    sf = torch.empty(B, H, D, D, dtype=torch.float32, device=q_raw.device) if output_final_state else None
    if workspace is None:
        workspace = torch.empty(cam_prep_scan_workspace_bytes(B, N, H, D, F, dt), dtype=torch.uint8,
                                device=q_raw.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_CAM_REVERSE if reverse else 0)
    st = load().cam_prep_scan_fwd(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(q_norm_w), _ptr(k_norm_w),
                                  _ptr(proj_q), _ptr(proj_kv), float(rope_base), _ptr(beta), _ptr(decay),
                                  _ptr(initial_state), _ptr(o), _ptr(sf), B, N, H, D, F, float(k_scale), float(eps),
                                  float(scale), flags, code, _ptr(workspace), ws_bytes, _stream(stream))
    _raise("cam_prep_scan_fwd", st)
    return o, sf


def cam_prep_fwd(q_raw, k_raw, v_raw, proj_q, proj_kv, q_norm_w=None, k_norm_w=None, rope_cos=None,
                 rope_sin=None, rope_base=10000.0, k_scale=0.5, eps=1e-6, with_norms=True, outs=None,
                 stream=None):
    """Fused camera prep.  Raw q,k,v [B,N,H,D] -> q,k,v [B,H,N,D] plus
    ||k||^2 before / after the projection and rotation, [B,H,N] fp32."""
    B, N, H, D = q_raw.shape
    dt = q_raw.dtype
    code = _dtype_code(q_raw)
    for name, t in (("q_raw", q_raw), ("k_raw", k_raw), ("v_raw", v_raw)):
        _check(t, name, (B, N, H, D), dt)
    _check(proj_q, "proj_q", (B, N, 4, 4), torch.float32)
    _check(proj_kv, "proj_kv", (B, N, 4, 4), torch.float32)
    for name, t in (("q_norm_w", q_norm_w), ("k_norm_w", k_norm_w)):
        if t is not None:
            _check(t, name, (H * D,), torch.float32)
    for name, t in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
        if t is not None:
            _check(t, name, (N, D // 2), torch.float32)
    dev = q_raw.device
    if outs is None:
        outs = tuple(torch.empty(B, H, N, D, dtype=dt, device=dev) for _ in range(3))
    pre = torch.empty(B, H, N, dtype=torch.float32, device=dev) if with_norms else None
    post = torch.empty(B, H, N, dtype=torch.float32, device=dev) if with_norms else None
    st = load().cam_prep_fwd(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(q_norm_w), _ptr(k_norm_w),
                             _ptr(proj_q), _ptr(proj_kv), _ptr(rope_cos), _ptr(rope_sin),
                             float(rope_base), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(pre),
                             _ptr(post), B, N, H, D, float(k_scale), float(eps), code, _stream(stream))
    _raise("cam_prep_fwd", st)
    return outs[0], outs[1], outs[2], pre, post


def cam_scan_bwd(q, k, v, beta, decay, do, initial_state=None, dfinal_state=None, scale=1.0, l2norm=False,
                 need_dinitial=False, workspace=None, stream=None, simt=False):
    """Backward of cam_scan_fwd (forward direction).  Returns (dq, dk, dv,
    dbeta, ddecay, dinitial_state or None); dq, dk, dv in the inputs' dtype,
    the rest fp32.  simt=True keeps the token gradients on the CUDA cores."""
    B, H, N, Dk = q.shape
    Dv = v.shape[-1]
    F = decay.shape[-1]
    if F <= 0 or N % F != 0:
        raise ValueError(f"{N} tokens do not split into {F} frames")
    S = N // F
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, N, Dk), dt)
    _check(k, "k", (B, H, N, Dk), dt)
    _check(v, "v", (B, H, N, Dv), dt)
    _check(beta, "beta", (B, H, N), dt)
    _check(decay, "decay", (B, H, F), torch.float32)
    _check(do, "do", (B, H, N, Dv), dt)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _check(t, name, (B, H, Dk, Dv), torch.float32)
    dev = q.device
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dv = torch.empty_like(v)
    dbeta = torch.empty(B, H, N, dtype=torch.float32, device=dev)
    ddecay = torch.empty(B, H, F, dtype=torch.float32, device=dev)
    ds0 = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev) if need_dinitial else None
    lib = load()
    need = lib.cam_scan_bwd_workspace_bytes(B, H, F, S, Dk, Dv, code)
    if workspace is None:
        workspace = torch.empty(int(need), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.cam_scan_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(decay), _ptr(initial_state), _ptr(do),
                          _ptr(dfinal_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(ddecay), _ptr(ds0),
                          B, H, F, S, Dk, Dv, float(scale),
                          (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0), code,
                          _ptr(workspace), ws_bytes, _stream(stream))
    _raise("cam_scan_bwd", st)
    return dq, dk, dv, dbeta, ddecay, ds0


def gdn_chunk_bwd_workspace_bytes(B, H, T, Dk, Dv, dtype=torch.bfloat16, r=1):
    code = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(load().gdn_chunk_bwd_workspace_bytes(B, H, T, r, Dk, Dv, code))


def deltaproduct_chunk_bwd(q, k, v, beta, g, do, initial_state=None, dfinal_state=None, scale=1.0, l2norm=False,
                           need_dinitial=False, workspace=None, stream=None, simt=False):
    """Backward of deltaproduct_chunk_fwd: k [B,H,T,r,Dk], v [B,H,T,r,Dv],
    beta [B,H,T,r].  Returns (dq, dk, dv, dbeta, dg, dinitial_state or None);
    dq, dk, dv in the inputs' dtype, the rest fp32."""
    B, H, T, Dk = q.shape
    r, Dv = k.shape[3], v.shape[-1]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, T, Dk), dt)
    _check(k, "k", (B, H, T, r, Dk), dt)
    _check(v, "v", (B, H, T, r, Dv), dt)
    _check(beta, "beta", (B, H, T, r), dt)
    _check(g, "g", (B, H, T), torch.float32)
    _check(do, "do", (B, H, T, Dv), dt)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _check(t, name, (B, H, Dk, Dv), torch.float32)
    dev = q.device
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta = torch.empty(B, H, T, r, dtype=torch.float32, device=dev)
    dg = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    ds0 = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev) if need_dinitial else None
    lib = load()
    if workspace is None:
        need = lib.gdn_chunk_bwd_workspace_bytes(B, H, T, r, Dk, Dv, code)
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0)
    st = lib.deltaproduct_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(initial_state), _ptr(do),
                                    _ptr(dfinal_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dg),
                                    _ptr(ds0), B, H, T, r, Dk, Dv, float(scale), flags,
                                    code,
                                    _ptr(workspace), ws_bytes, _stream(stream))
    _raise("deltaproduct_chunk_bwd", st)
    return dq, dk, dv, dbeta, dg, ds0


def masked_deltaproduct_chunk_bwd(q, k, v, beta, g, mask, do, initial_state=None, dfinal_state=None, scale=1.0,
                                  l2norm=False, need_dinitial=False, workspace=None, stream=None, simt=False):
    """Backward of masked_deltaproduct_chunk_fwd.  Returns (dq, dk, dv, dbeta,
    dg, dinitial_state or None); dq, dk, dv in the inputs' dtype, the rest fp32."""
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    r = mask.shape[0]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, T, Dk), dt)
    _check(k, "k", (B, H, T, Dk), dt)
    _check(v, "v", (B, H, T, Dv), dt)
    _check(beta, "beta", (B, H, T), dt)
    _check(g, "g", (B, H, T), torch.float32)
    _check(mask, "mask", (r, r), torch.float32)
    _check(do, "do", (B, H, T, Dv), dt)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _check(t, name, (B, H, Dk, Dv), torch.float32)
    dev = q.device
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    dg = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    ds0 = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev) if need_dinitial else None
    lib = load()
    if workspace is None:
        need = lib.masked_deltaproduct_chunk_bwd_workspace_bytes(B, H, T, r, Dk, Dv, code)
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0)
    st = lib.masked_deltaproduct_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(mask),
                                           _ptr(initial_state), _ptr(do), _ptr(dfinal_state), _ptr(dq), _ptr(dk),
                                           _ptr(dv), _ptr(dbeta), _ptr(dg), _ptr(ds0), B, H, T, r, Dk, Dv,
                                           float(scale), flags,
                                           code, _ptr(workspace),
                                           ws_bytes, _stream(stream))
    _raise("masked_deltaproduct_chunk_bwd", st)
    return dq, dk, dv, dbeta, dg, ds0


def gdn_chunk_bwd(q, k, v, beta, g, do, initial_state=None, dfinal_state=None, scale=1.0, l2norm=False,
                  need_dinitial=False, workspace=None, stream=None, simt=False):
    """Backward of gdn_chunk_fwd.  Returns (dq, dk, dv, dbeta, dg,
    dinitial_state or None); dq, dk, dv in the inputs' dtype, the rest fp32."""
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    dt = q.dtype
    code = _dtype_code(q)
    _check(q, "q", (B, H, T, Dk), dt)
    _check(k, "k", (B, H, T, Dk), dt)
    _check(v, "v", (B, H, T, Dv), dt)
    _check(beta, "beta", (B, H, T), dt)
    _check(g, "g", (B, H, T), torch.float32)
    _check(do, "do", (B, H, T, Dv), dt)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _check(t, name, (B, H, Dk, Dv), torch.float32)
    dev = q.device
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dbeta = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    dg = torch.empty(B, H, T, dtype=torch.float32, device=dev)
    ds0 = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev) if need_dinitial else None
    lib = load()
    if workspace is None:
        need = lib.gdn_chunk_bwd_workspace_bytes(B, H, T, 1, Dk, Dv, code)
        workspace = torch.empty(max(int(need), 16), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_PATH_SIMT if simt else 0)
    st = lib.gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(initial_state), _ptr(do),
                           _ptr(dfinal_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dg), _ptr(ds0), B, H, T,
                           Dk, Dv, float(scale), flags,
                           code, _ptr(workspace), ws_bytes, _stream(stream))
    _raise("gdn_chunk_bwd", st)
    return dq, dk, dv, dbeta, dg, ds0


def cam_prep_bwd(q_raw, k_raw, proj_q, proj_kv, dq_out, dk_out, dv_out, dk_pre_sq=None, dk_post_sq=None,
                 q_norm_w=None, k_norm_w=None, rope_cos=None, rope_sin=None, rope_base=10000.0, k_scale=0.5,
                 eps=1e-6, stream=None):
    """Backward of cam_prep_fwd: gradients of the raw q, k, v [B,N,H,D] from
    those of q_out, k_out, v_out [B,H,N,D] (and of k_pre_sq, k_post_sq)."""
    B, N, H, D = q_raw.shape
    dt = q_raw.dtype
    code = _dtype_code(q_raw)
    _check(k_raw, "k_raw", (B, N, H, D), dt)
    _check(proj_q, "proj_q", (B, N, 4, 4), torch.float32)
    _check(proj_kv, "proj_kv", (B, N, 4, 4), torch.float32)
    for name, t in (("dq_out", dq_out), ("dk_out", dk_out), ("dv_out", dv_out)):
        _check(t, name, (B, H, N, D), dt)
    for name, t in (("dk_pre_sq", dk_pre_sq), ("dk_post_sq", dk_post_sq)):
        if t is not None:
            _check(t, name, (B, H, N), torch.float32)
    outs = tuple(torch.empty(B, N, H, D, dtype=dt, device=q_raw.device) for _ in range(3))
    st = load().cam_prep_bwd(_ptr(q_raw), _ptr(k_raw), _ptr(q_norm_w), _ptr(k_norm_w), _ptr(proj_q), _ptr(proj_kv),
                             _ptr(rope_cos), _ptr(rope_sin), float(rope_base), _ptr(dq_out), _ptr(dk_out),
                             _ptr(dv_out), _ptr(dk_pre_sq), _ptr(dk_post_sq), _ptr(outs[0]), _ptr(outs[1]),
                             _ptr(outs[2]), B, N, H, D, float(k_scale), float(eps), code, _stream(stream))
    _raise("cam_prep_bwd", st)
    return outs


# ------------------------------------------------- around a linear-attention layer
# (a decoding step's kernels take a few microseconds: these calls keep to plain
# attribute reads, and ask for a workspace's size once for each set of sizes)
_NO_BYTES = ctypes.c_size_t(-1).value


def _dense(t, name, shape, dtype):
    """_check, for the case that all is well."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        _check(t, name, shape, dtype)


def _at(stream, t):
    """The raw stream of a call: the given one or the current one of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.device.index) if stream is None else stream.cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _bytes(fn, *sizes):
    """A workspace query's answer."""
    need = getattr(load(), fn)(*sizes)
    if need == _NO_BYTES:
        raise ValueError(f"sizes rejected by {fn}")
    return int(need)


def _scratch(need, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _room(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _strided(t, name, shape, dtype):
    """As _check for a tensor whose last dimension is contiguous and whose
    other strides are multiples of 16 bytes; whether it is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return True
    size = t.element_size()
    for n, s in zip(t.shape[:-1], t.stride()[:-1]):
        if n > 1 and s * size % 16 != 0:
            raise ValueError(f"{name}'s strides {t.stride()} must be multiples of 16 bytes")
    if t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return False


def _gates(g, shape):
    """Checks log-decays [B,H,T] (any strides) or [H]: (per head, contiguous)."""
    if isinstance(g, torch.Tensor) and g.dim() == 1:
        _dense(g, "g", (shape[1],), torch.float32)
        return True, True
    if not isinstance(g, torch.Tensor) or not g.is_cuda:
        raise TypeError("g must be a CUDA tensor")
    if g.shape != shape:
        raise ValueError(f"g has shape {tuple(g.shape)}, expected {shape} or ({shape[1]},)")
    if g.dtype is not torch.float32:
        raise TypeError(f"g must be torch.float32, got {g.dtype}")
    return False, g.is_contiguous()


def _steps(*tensors):
    """The strides array of linattn_chunk_*: (batch, head, token) of each; a
    dimension of one element has none that matters."""
    out = []
    for t in tensors:
        if t.dim() == 1:
            out += (0, 0, 0)
        else:
            out += [s if n > 1 else 0 for n, s in zip(t.shape[:3], t.stride())]
    return (ctypes.c_longlong * 15)(*out)


_HERE = contextlib.nullcontext()


def _on(stream):
    """Allocations of a call belong to the stream that it runs on."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _expanded(t):
    return any(s == 0 and n > 1 for n, s in zip(t.shape, t.stride()))


def _overlaps(t):
    """Whether elements may share memory (an expanded tensor, sliding windows):
    a dimension steps by less than those of smaller steps span."""
    span = 1
    for s, n in sorted((s, n) for n, s in zip(t.shape, t.stride()) if n > 1):
        if s < span:
            return True
        span += s * (n - 1)
    return False


def _linattn_sizes(q, k, v, g, cu_seqlens, initial_state):
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor) or q.dim() != 4 or v.dim() != 4:
        raise TypeError("q, k and v must be [B,heads,T,D] CUDA tensors")
    B, Hk, T, Dk = q.shape
    _, H, _, Dv = v.shape
    code = _dtype_code(q)
    dense = _strided(q, "q", (B, Hk, T, Dk), q.dtype)
    dense = _strided(k, "k", (B, Hk, T, Dk), q.dtype) and dense
    dense = _strided(v, "v", (B, H, T, Dv), q.dtype) and dense
    per_head, plain = _gates(g, (B, H, T))
    if Hk == 0 or H % Hk != 0:
        raise ValueError(f"{Hk} query / key heads do not divide {H} value heads")
    n_seq = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold at least two offsets")
        _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32)
        if B != 1:
            raise ValueError("packed sequences (cu_seqlens) lie in one row: B must be 1")
        n_seq = cu_seqlens.numel() - 1
    if initial_state is not None:
        _dense(initial_state, "initial_state", (n_seq, H, Dk, Dv), torch.float32)
    return B, H, Hk, T, Dk, Dv, n_seq, code, per_head, dense and plain


def linattn_chunk_fwd(q, k, v, g, initial_state=None, output_final_state=False, cu_seqlens=None, scale=1.0, o=None,
                      workspace=None, stream=None, simt=False):
    """Linear attention with a decay for each head over prompts.  q, k
    [B,Hk,T,Dk]; v [B,H,T,Dv] (all bf16 or all fp32, last dimension
    contiguous); g [B,H,T] or [H] fp32 log-decays.  cu_seqlens: int32 CUDA
    offsets of sequences packed into one row (a token-major [T,H,D] tensor x
    goes in as x.unsqueeze(0).transpose(1, 2)).  initial_state
    [sequences,H,Dk,Dv] fp32.  Returns (o, final_state or None); o has v's
    strides unless it is given.  In bf16, o's last bit may depend on whether a
    final state is asked for."""
    if o is None and workspace is None and stream is None:
        r = (_front or _quick()).fwd(q, k, v, g, initial_state, output_final_state, cu_seqlens, scale, simt)
        if r is not NotImplemented:
            return r
    B, H, Hk, T, Dk, Dv, n_seq, code, per_head, dense = _linattn_sizes(q, k, v, g, cu_seqlens, initial_state)
    flags = (GDN_G_PER_HEAD if per_head else 0) | (GDN_PATH_SIMT if simt else 0)
    need = _bytes("linattn_chunk_fwd_workspace_bytes", B, H, Hk, T, Dk, Dv, n_seq, cu_seqlens is not None, flags, code)
    with _on(stream):
        if not dense:
            q, k, v = (t.contiguous() if _expanded(t) else t for t in (q, k, v))
        if o is None:
            o = torch.empty_like(v)
            dense = dense and o.is_contiguous()
        else:
            dense = _strided(o, "o", (B, H, T, Dv), q.dtype) and dense
        sf = torch.empty(n_seq, H, Dk, Dv, dtype=torch.float32, device=q.device) if output_final_state else None
        if workspace is None:
            workspace = _scratch(need, q.device)
    st = load().linattn_chunk_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(initial_state),
                                  o.data_ptr(), _addr(sf), _addr(cu_seqlens), None if dense else _steps(q, k, v, o, g),
                                  n_seq, B, H, Hk, T, Dk, Dv, scale, flags, code, _addr(workspace), _room(workspace),
                                  _at(stream, q))
    if st:
        _raise("linattn_chunk_fwd", st)
    return o, sf


def linattn_chunk_bwd(q, k, v, g, dout, initial_state=None, dfinal_state=None, cu_seqlens=None, scale=1.0,
                      workspace=None, stream=None, simt=False):
    """Backward of linattn_chunk_fwd.  dout [B,H,T,Dv], dfinal_state
    [sequences,H,Dk,Dv] fp32.  Returns (dq, dk, dv, dg, dinitial_state or
    None): the first three in the tensors' type, dg fp32 in g's shape (its sum
    over batch and tokens for g [H]).  Gradients are allocated with their
    tensors' strides: those of slices of one projection take its memory each.
    The workspace, if not given, is 12 bytes (fp32: 16) for each Dk*Dv of every
    128 tokens and value head, and 8*Dk for each token and value head of shared
    heads."""
    if workspace is None and stream is None:
        r = (_front or _quick()).bwd(q, k, v, g, dout, initial_state, dfinal_state, cu_seqlens, scale, simt)
        if r is not NotImplemented:
            return r
    B, H, Hk, T, Dk, Dv, n_seq, code, per_head, dense = _linattn_sizes(q, k, v, g, cu_seqlens, initial_state)
    dense = _strided(dout, "dout", (B, H, T, Dv), q.dtype) and dense
    if dfinal_state is not None:
        _dense(dfinal_state, "dfinal_state", (n_seq, H, Dk, Dv), torch.float32)
    flags = (GDN_G_PER_HEAD if per_head else 0) | (GDN_PATH_SIMT if simt else 0)
    need = _bytes("linattn_chunk_bwd_workspace_bytes", B, H, Hk, T, Dk, Dv, n_seq, cu_seqlens is not None, flags, code)
    with _on(stream):
        if not dense:
            # gradients take their tensors' strides, so those may not overlap
            q, k, v, g = (t.contiguous() if _overlaps(t) else t for t in (q, k, v, g))
            dout = dout.contiguous() if _expanded(dout) else dout
        dq, dk, dv, dg = (torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device) for t in (q, k, v, g))
        ds0 = torch.empty_like(initial_state) if initial_state is not None else None
        if workspace is None:
            workspace = _scratch(need, q.device)
    st = load().linattn_chunk_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _addr(initial_state),
                                  dout.data_ptr(), _addr(dfinal_state), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                  dg.data_ptr(), _addr(ds0), _addr(cu_seqlens),
                                  None if dense else _steps(q, k, v, dout, g), n_seq, B, H, Hk, T, Dk, Dv, scale, flags,
                                  code, _addr(workspace), _room(workspace), _at(stream, q))
    if st:
        _raise("linattn_chunk_bwd", st)
    return dq, dk, dv, dg, ds0


def _step(fn_name, q, k, v, beta, g, state, slots, state_out, scale, l2norm, o, stream):
    if o is None and stream is None:
        r = (_front or _quick()).step(q, k, v, beta, g, state, slots, state_out, scale, l2norm)
        if r is not NotImplemented:
            return r
    B, Hk, Dk = q.shape
    _, H, Dv = v.shape
    n_slots = state.shape[0]
    dt = q.dtype
    code = _dtype_code(q)
    _dense(q, "q", (B, Hk, Dk), dt)
    _dense(k, "k", (B, Hk, Dk), dt)
    _dense(v, "v", (B, H, Dv), dt)
    if Hk == 0 or H % Hk != 0:
        raise ValueError(f"{Hk} query / key heads do not divide {H} value heads")
    per_head = g.dim() == 1
    _dense(g, "g", (H,) if per_head else (B, H), torch.float32)
    _dense(state, "state", (n_slots, H, Dk, Dv), torch.float32)
    if state_out is None:
        state_out = state
    elif state_out is not state:
        _dense(state_out, "state_out", (n_slots, H, Dk, Dv), torch.float32)
    if slots is not None:
        _dense(slots, "slots", (B,), torch.int32)
    elif B > n_slots:
        raise ValueError(f"{B} rows but {n_slots} pages")
    if o is None:
        with _on(stream):
            o = torch.empty_like(v)
    else:
        _dense(o, "o", (B, H, Dv), dt)
    flags = (GDN_G_PER_HEAD if per_head else 0) | (GDN_QK_L2NORM if l2norm else 0)
    rest = (g.data_ptr(), state.data_ptr(), state_out.data_ptr(), _addr(slots), o.data_ptr(), B, H, Hk, Dk, Dv, n_slots,
            scale, flags, code, _at(stream, q))
    if beta is None:
        st = load().linattn_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), *rest)
    else:
        _dense(beta, "beta", (B, H), dt)
        st = load().gdn_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), *rest)
    if st:
        _raise(fn_name, st)
    return o


def linattn_step(q, k, v, g, state, slots=None, state_out=None, scale=1.0, o=None, stream=None):
    """One token of linear attention with a decay for each head.  q, k
    [B,Hk,Dk]; v [B,H,Dv]; g [B,H] or [H] fp32; state [slots,H,Dk,Dv] fp32,
    updated in place unless state_out is given; slots int32 [B]: each row's
    page, -1 for an idle row (o = 0).  Returns o [B,H,Dv]."""
    return _step("linattn_step", q, k, v, None, g, state, slots, state_out, scale, False, o, stream)


def gdn_step(q, k, v, beta, g, state, slots=None, state_out=None, scale=1.0, l2norm=False, o=None, stream=None):
    """One token of the gated delta rule (gdn_chunk_fwd's recurrence) against a
    pool of states; beta [B,H], the rest as linattn_step."""
    if beta is None:
        raise TypeError("beta must be a CUDA tensor (the step without the delta rule is linattn_step)")
    return _step("gdn_step", q, k, v, beta, g, state, slots, state_out, scale, l2norm, o, stream)


def rms_norm_fwd(x, weight=None, residual=None, eps=1e-6, out_dtype=None, group=0, stream=None):
    """h = x + residual and its root-mean-square norm over the last dimension.
    out_dtype: None (x's) or torch.float8_e4m3fn, then with scales [...,C/group]
    (group 32, 64 or 128) or [...,1] (group 0: one a row).  Returns (y, scales or
    None, h); h is x itself without a residual."""
    e4m3 = out_dtype is torch.float8_e4m3fn
    if stream is None and (e4m3 or out_dtype is None):
        r = (_front or _quick()).norm(x, weight, residual, eps, e4m3, group)
        if r is not NotImplemented:
            return r
    C = x.shape[-1]
    code = _dtype_code(x)
    _dense(x, "x", x.shape, x.dtype)
    if residual is not None:
        _dense(residual, "residual", x.shape, x.dtype)
    if weight is not None:
        _dense(weight, "weight", (C,), torch.float32)
    if not e4m3 and out_dtype not in (None, x.dtype):
        raise TypeError(f"out_dtype must be {x.dtype} or torch.float8_e4m3fn, got {out_dtype}")
    if group and (not e4m3 or group not in (32, 64, 128) or C % group):
        raise ValueError(f"group {group}: 32, 64 or 128 dividing the last dimension, with an e4m3 output")
    scales = None
    with _on(stream):
        y = torch.empty_like(x, dtype=out_dtype)
        if e4m3:
            scales = torch.empty((*x.shape[:-1], C // group if group else 1), dtype=torch.float32, device=x.device)
        h = torch.empty_like(x) if residual is not None else x
    rows = x.numel() // C if C else 0
    st = load().rms_norm_fwd(x.data_ptr(), _addr(residual), _addr(weight), y.data_ptr(), _addr(scales),
                             h.data_ptr() if residual is not None else None, rows, C, group, eps, e4m3, code,
                             _at(stream, x))
    if st:
        _raise("rms_norm_fwd", st)
    return y, scales, h


def rms_norm_bwd(dy, h, weight=None, dresidual=None, eps=1e-6, workspace=None, stream=None):
    """Backward of rms_norm_fwd at the h that it returned: (dx, dweight [C]
    fp32).  dresidual: the gradient that reaches h past the norm; dx is also
    the residual's gradient."""
    if workspace is None and stream is None:
        r = (_front or _quick()).norm_back(dy, h, weight, dresidual, eps)
        if r is not NotImplemented:
            return r
    C = h.shape[-1]
    code = _dtype_code(h)
    _dense(h, "h", h.shape, h.dtype)
    _dense(dy, "dy", h.shape, h.dtype)
    if dresidual is not None:
        _dense(dresidual, "dresidual", h.shape, h.dtype)
    if weight is not None:
        _dense(weight, "weight", (C,), torch.float32)
    rows = h.numel() // C if C else 0
    need = _bytes("rms_norm_bwd_workspace_bytes", rows, C)
    with _on(stream):
        dx = torch.empty_like(h)
        dw = torch.empty(C, dtype=torch.float32, device=h.device)
        if workspace is None:
            workspace = _scratch(need, h.device)
    st = load().rms_norm_bwd(dy.data_ptr(), h.data_ptr(), _addr(weight), _addr(dresidual), dx.data_ptr(), dw.data_ptr(),
                             rows, C, eps, code, _addr(workspace), _room(workspace), _at(stream, h))
    if st:
        _raise("rms_norm_bwd", st)
    return dx, dw


def _pool(pool):
    """(layers, slots, page bytes) of a contiguous [layers,slots,...] pool."""
    if not isinstance(pool, torch.Tensor) or not pool.is_cuda:
        raise TypeError("pool must be a CUDA tensor")
    if pool.dim() < 2 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous [layers,slots,...] tensor")
    layers, n_slots = pool.shape[:2]
    page = pool.stride(1) * pool.element_size() if pool.numel() else 0
    if page % 16:
        raise ValueError(f"a page of {page} bytes is not a multiple of 16")
    return layers, n_slots, page


def _slots(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise TypeError(f"{name} must be a one-dimensional CUDA tensor")
    _dense(t, name, t.shape, torch.int32)
    return t.numel()


def state_pool_copy(pool, src, dst, stream=None):
    """pool[:, dst[i]] = pool[:, src[i]] (zeros for src -1); indices out of
    range are skipped.  Destinations are distinct and no one's source."""
    layers, n_slots, page = _pool(pool)
    n = _slots(src, "src")
    if _slots(dst, "dst") != n:
        raise ValueError(f"{n} sources but {dst.numel()} destinations")
    st = load().state_pool_copy(pool.data_ptr(), layers, n_slots, page, src.data_ptr(), dst.data_ptr(), n,
                                _at(stream, pool))
    if st:
        _raise("state_pool_copy", st)


def state_pool_fork(pool, live, parents, stream=None):
    """Gives each parent (a live slot, or -1 for a new request's page of zeros)
    the lowest free slot, with a copy of its page in every layer of pool
    [layers,slots,...].  live uint8 [slots] is updated.  Returns the children,
    int32, -1 where the parent is not live or no slot is left."""
    if stream is None:
        r = (_front or _quick()).fork(pool, live, parents)
        if r is not NotImplemented:
            return r
    layers, n_slots, page = _pool(pool)
    _dense(live, "live", (n_slots,), torch.uint8)
    n = _slots(parents, "parents")
    need = _bytes("state_pool_fork_workspace_bytes", n_slots, n)
    with _on(stream):
        children = torch.empty_like(parents)
        ws = _scratch(need, pool.device)
    st = load().state_pool_fork(pool.data_ptr(), layers, n_slots, page, live.data_ptr(), parents.data_ptr(),
                                children.data_ptr(), n, _addr(ws), need, _at(stream, pool))
    if st:
        _raise("state_pool_fork", st)
    return children


def state_pool_free(live, slots, stream=None):
    """Marks slots (int32; out-of-range ones are skipped) free in live uint8."""
    _dense(live, "live", live.shape, torch.uint8)
    n = _slots(slots, "slots")
    st = load().state_pool_free(live.data_ptr(), live.numel(), slots.data_ptr(), n, _at(stream, live))
    if st:
        _raise("state_pool_free", st)


def state_pool_compact(pool, live, stream=None):
    """Moves the live pages of pool [layers,slots,...] into its first slots and
    updates live.  Returns (remap, n_live): int32 [slots], each slot's new
    place or -1, and the count, int32 [1], on the device."""
    if stream is None:
        r = (_front or _quick()).compact(pool, live)
        if r is not NotImplemented:
            return r
    layers, n_slots, page = _pool(pool)
    _dense(live, "live", (n_slots,), torch.uint8)
    need = _bytes("state_pool_compact_workspace_bytes", n_slots)
    with _on(stream):
        remap = torch.empty(n_slots, dtype=torch.int32, device=pool.device)
        n_live = torch.empty(1, dtype=torch.int32, device=pool.device)
        ws = _scratch(need, pool.device)
    st = load().state_pool_compact(pool.data_ptr(), layers, n_slots, page, live.data_ptr(), remap.data_ptr(),
                                   n_live.data_ptr(), _addr(ws), need, _at(stream, pool))
    if st:
        _raise("state_pool_compact", st)
    return remap, n_live


# ------------------------------------------------- next to a mixer
def _same_device(like, *tensors):
    """All tensors of a call lie on one device."""
    for t in tensors:
        if t is not None and t.device != like.device:
            raise ValueError(f"tensors on {like.device} and {t.device}: a call's tensors lie on one device")


@contextlib.contextmanager
def _device(t, stream):
    """The device of a call's tensors is the current one while it launches, and its
    allocations belong to the stream that it runs on."""
    with torch.cuda.device(t.device), _on(stream):
        yield


def _pitches(*tensors):
    """A strides array: those of every dimension but the last; a dimension of one
    element has none that matters."""
    out = []
    for t in tensors:
        out += [s if n > 1 else 0 for n, s in zip(t.shape[:-1], t.stride())]
    return (ctypes.c_longlong * len(out))(*out)


def _rows_of(x, name, cu_seqlens, C=None):
    """(B, T, C, sequences) of [B,T,C] rows."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise TypeError(f"{name} must be a [B,T,channels] CUDA tensor")
    B, T, C = x.shape
    n_seq = B
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must hold at least two offsets")
        _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32)
        if B != 1:
            raise ValueError("packed sequences (cu_seqlens) lie in one row: B must be 1")
        n_seq = cu_seqlens.numel() - 1
    return B, T, C, n_seq


def _maybe(t, name, shape, dtype):
    if t is not None:
        _dense(t, name, shape, dtype)


def _written(t, name, shape, dtype):
    """As _strided, for an output of the caller's: no two elements in one place."""
    _strided(t, name, shape, dtype)
    if _overlaps(t):
        raise ValueError(f"{name}'s elements share memory")


def _side_by_side(a, b):
    """Whether the rows of a and b (their last dimensions) are columns of one buffer's
    rows: all begin at one of two places in what their strides are multiples of."""
    every = math.gcd(*(s * t.element_size() for t in (a, b) for n, s in zip(t.shape[:-1], t.stride()) if n > 1))
    wide = lambda t: t.shape[-1] * t.element_size()  # noqa: E731
    return every > 0 and wide(a) <= (b.data_ptr() - a.data_ptr()) % every <= every - wide(b)


def _apart(a, b, names):
    """A call reads b after it has begun to write a: they may not share memory."""
    if a is not None and b is not None and a.numel() and b.numel():
        span = lambda t: t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()  # noqa: E731
        if a.data_ptr() < span(b) and b.data_ptr() < span(a) and not _side_by_side(a, b):
            raise ValueError(f"{names} share memory")


def _taps(weight, bias, C):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise TypeError("weight must be a [channels,W] CUDA tensor")
    W = weight.shape[1]
    _dense(weight, "weight", (C, W), torch.float32)
    _maybe(bias, "bias", (C,), torch.float32)
    return W


def causal_conv_fwd(x, weight, bias=None, initial_window=None, output_final_window=False, cu_seqlens=None, silu=True,
                    y=None, stream=None):
    """The short causal convolution of each channel, then SiLU (or not).  x [B,T,C]
    (bf16 or fp32, channels contiguous, C a multiple of 8 or 4); weight [C,W] fp32,
    W 2 to 4, the last tap the token's own; bias [C] fp32.  initial_window
    [sequences,W-1,C], the inputs before each sequence; cu_seqlens as in
    linattn_chunk_fwd.  Returns (y, final_window or None): the last W-1 inputs of
    each sequence, counted over its window and its tokens."""
    if y is None and stream is None:
        r = (_front or _quick()).conv(x, weight, bias, initial_window, output_final_window, cu_seqlens, silu)
        if r is not NotImplemented:
            return r
    B, T, C, n_seq = _rows_of(x, "x", cu_seqlens)
    code, W = _dtype_code(x), _taps(weight, bias, C)
    _strided(x, "x", (B, T, C), x.dtype)
    _maybe(initial_window, "initial_window", (n_seq, W - 1, C), x.dtype)
    _same_device(x, weight, bias, initial_window, cu_seqlens, y)
    with _device(x, stream):
        if y is None:
            y = torch.empty(B, T, C, dtype=x.dtype, device=x.device)
        else:
            _written(y, "y", (B, T, C), x.dtype)
            _apart(y, x, "x and y")
            _apart(y, initial_window, "initial_window and y")
        win = torch.empty(n_seq, W - 1, C, dtype=x.dtype, device=x.device) if output_final_window else None
        st = load().causal_conv_fwd(x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(initial_window), y.data_ptr(),
                                    _addr(win), _addr(cu_seqlens), _pitches(x, y), n_seq, B, T, C, W,
                                    GDN_SILU if silu else 0, code, _at(stream, x))
    if st:
        _raise("causal_conv_fwd", st)
    return y, win


def causal_conv_bwd(x, weight, dy, bias=None, initial_window=None, dfinal_window=None, cu_seqlens=None, silu=True,
                    workspace=None, stream=None):
    """Backward of causal_conv_fwd.  dy [B,T,C], dfinal_window [sequences,W-1,C] in
    x's type.  Returns (dx, dweight [C,W] fp32, dbias [C] fp32 or None without a
    bias, dinitial_window or None without an initial window)."""
    if workspace is None and stream is None:
        r = (_front or _quick()).conv_back(x, weight, dy, bias, initial_window, dfinal_window, cu_seqlens, silu)
        if r is not NotImplemented:
            return r
    B, T, C, n_seq = _rows_of(x, "x", cu_seqlens)
    code, W = _dtype_code(x), _taps(weight, bias, C)
    _strided(x, "x", (B, T, C), x.dtype)
    _strided(dy, "dy", (B, T, C), x.dtype)
    _maybe(initial_window, "initial_window", (n_seq, W - 1, C), x.dtype)
    _maybe(dfinal_window, "dfinal_window", (n_seq, W - 1, C), x.dtype)
    _same_device(x, weight, dy, bias, initial_window, dfinal_window, cu_seqlens, workspace)
    need = _bytes("causal_conv_bwd_workspace_bytes", B, T, C, W)
    with _device(x, stream):
        dx = torch.empty(B, T, C, dtype=x.dtype, device=x.device)
        dw = torch.empty(C, W, dtype=torch.float32, device=x.device)
        db = torch.empty(C, dtype=torch.float32, device=x.device) if bias is not None else None
        dwin = torch.empty_like(initial_window) if initial_window is not None else None
        if workspace is None:
            workspace = _scratch(need, x.device)
        st = load().causal_conv_bwd(x.data_ptr(), weight.data_ptr(), _addr(bias), dy.data_ptr(), _addr(initial_window),
                                    _addr(dfinal_window), dx.data_ptr(), dw.data_ptr(), _addr(db), _addr(dwin),
                                    _addr(cu_seqlens), _pitches(x, dy), n_seq, B, T, C, W, GDN_SILU if silu else 0, code,
                                    _addr(workspace), _room(workspace), _at(stream, x))
    if st:
        _raise("causal_conv_bwd", st)
    return dx, dw, db, dwin


def _row(t, name, shape, dtype):
    """A [B,n] tensor whose rows may lie apart."""
    _strided(t, name, shape, dtype)
    return t.stride(0) if shape[0] > 1 else 0


def _pages(pool, name, shape, dtype, slots, B):
    """Checks a pool [slots,...] and the rows' slots; how many pages it has."""
    if not isinstance(pool, torch.Tensor) or pool.dim() != 1 + len(shape):
        raise TypeError(f"{name} must be a [slots,{','.join(map(str, shape))}] CUDA tensor")
    n = pool.shape[0]
    _dense(pool, name, (n, *shape), dtype)
    if slots is not None:
        _dense(slots, "slots", (B,), torch.int32)
    elif B > n:
        raise ValueError(f"{B} rows but {n} pages")
    return n


def causal_conv_step(x, weight, window, bias=None, slots=None, window_out=None, silu=True, y=None, stream=None):
    """One token of causal_conv_fwd for each row of x [B,C] (rows may lie apart)
    against a pool of windows [slots,W-1,C] in x's type, updated in place unless
    window_out is given; slots int32 [B]: each row's page, -1 for an idle row (y =
    0).  Returns y [B,C]."""
    if y is None and stream is None:
        r = (_front or _quick()).conv_step(x, weight, window, bias, slots, window_out, silu)
        if r is not NotImplemented:
            return r
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a [B,channels] CUDA tensor")
    B, C = x.shape
    code, W = _dtype_code(x), _taps(weight, bias, C)
    step = _row(x, "x", (B, C), x.dtype)
    n = _pages(window, "window", (W - 1, C), x.dtype, slots, B)
    if window_out is None:
        window_out = window
    elif window_out is not window:
        _dense(window_out, "window_out", window.shape, x.dtype)
        if window_out.data_ptr() != window.data_ptr():
            _apart(window_out, window, "window and window_out")
    _same_device(x, weight, window, bias, slots, window_out, y)
    with _device(x, stream):
        if y is None:
            y = torch.empty(B, C, dtype=x.dtype, device=x.device)
        else:
            _dense(y, "y", (B, C), x.dtype)
            for t, name in ((x, "x"), (window, "window"), (window_out, "window_out")):
                _apart(y, t, f"{name} and y")
        st = load().causal_conv_step(x.data_ptr(), weight.data_ptr(), _addr(bias), window.data_ptr(), window_out.data_ptr(),
                                     _addr(slots), y.data_ptr(), step, B, C, W, n, GDN_SILU if silu else 0, code,
                                     _at(stream, x))
    if st:
        _raise("causal_conv_step", st)
    return y


def _scan_sizes(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens):
    rows, T, Di, n_seq = _rows_of(x, "x", cu_seqlens)
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise TypeError("A must be a [channels,N] CUDA tensor")
    code, N = _dtype_code(x), A.shape[1]
    _dense(A, "A", (Di, N), torch.float32)
    for t, name, n in ((x, "x", Di), (dt, "dt", Di), (B, "B", N), (C, "C", N), (z, "z", Di)):
        if t is not None or name != "z":
            _strided(t, name, (rows, T, n), x.dtype)
    _maybe(D, "D", (Di,), torch.float32)
    _maybe(dt_bias, "dt_bias", (Di,), torch.float32)
    _maybe(initial_state, "initial_state", (n_seq, Di, N), torch.float32)
    _same_device(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens)
    return rows, T, Di, N, n_seq, code


def ssm_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_state=None, output_final_state=False,
                 cu_seqlens=None, softplus=True, y=None, workspace=None, stream=None):
    """The selective state space scan over prompts: with steps s = softplus(dt +
    dt_bias) (or their sum alone), h = exp(s A) h + s x B, y = (C.h + D x) silu(z).
    x, dt, z [B,T,Di], B, C [B,T,N] (all bf16 or all fp32, the last dimension
    contiguous, Di a multiple of 8 or 4, N 8, 16 or 32); A [Di,N], D, dt_bias [Di]
    fp32; initial_state [sequences,Di,N] fp32; cu_seqlens as in linattn_chunk_fwd.
    Returns (y, final_state or None)."""
    if y is None and workspace is None and stream is None:
        r = (_front or _quick()).scan(x, dt, A, B, C, D, z, dt_bias, initial_state, output_final_state, cu_seqlens, softplus)
        if r is not NotImplemented:
            return r
    rows, T, Di, N, n_seq, code = _scan_sizes(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens)
    _same_device(x, y, workspace)
    need = _bytes("ssm_scan_fwd_workspace_bytes", rows, T, Di, N, code)
    with _device(x, stream):
        if y is None:
            y = torch.empty(rows, T, Di, dtype=x.dtype, device=x.device)
        else:
            _written(y, "y", (rows, T, Di), x.dtype)
            for t, name in ((x, "x"), (dt, "dt"), (B, "B"), (C, "C"), (z, "z"), (initial_state, "initial_state")):
                _apart(y, t, f"{name} and y")
        sf = torch.empty(n_seq, Di, N, dtype=torch.float32, device=x.device) if output_final_state else None
        if workspace is None:
            workspace = _scratch(need, x.device)
        st = load().ssm_scan_fwd(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z),
                                 _addr(dt_bias), _addr(initial_state), y.data_ptr(), _addr(sf), _addr(cu_seqlens),
                                 _pitches(x, dt, B, C, x if z is None else z, y), n_seq, rows, T, Di, N,
                                 GDN_DT_SOFTPLUS if softplus else 0, code, _addr(workspace), _room(workspace),
                                 _at(stream, x))
    if st:
        _raise("ssm_scan_fwd", st)
    return y, sf


def ssm_scan_bwd(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, initial_state=None, dfinal_state=None,
                 cu_seqlens=None, softplus=True, workspace=None, stream=None):
    """Backward of ssm_scan_fwd.  dy [B,T,Di] in x's type, dfinal_state
    [sequences,Di,N] fp32.  Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias,
    dinitial_state), contiguous: those of tensors in their type, dA, dD, ddt_bias and
    dinitial_state in fp32; None for inputs that are not given.  The workspace, if
    not given, takes Di N bytes a token and more."""
    if workspace is None and stream is None:
        r = (_front or _quick()).scan_back(x, dt, A, B, C, dy, D, z, dt_bias, initial_state, dfinal_state, cu_seqlens, softplus)
        if r is not NotImplemented:
            return r
    rows, T, Di, N, n_seq, code = _scan_sizes(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens)
    _strided(dy, "dy", (rows, T, Di), x.dtype)
    _maybe(dfinal_state, "dfinal_state", (n_seq, Di, N), torch.float32)
    _same_device(x, dy, dfinal_state, workspace)
    need = _bytes("ssm_scan_bwd_workspace_bytes", rows, T, Di, N, code)
    with _device(x, stream):
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=x.device)  # noqa: E731
        dx, ddt = new((rows, T, Di), x.dtype), new((rows, T, Di), x.dtype)
        dB, dC = new((rows, T, N), x.dtype), new((rows, T, N), x.dtype)
        dA = new((Di, N), torch.float32)
        dD = new((Di,), torch.float32) if D is not None else None
        dz = new((rows, T, Di), x.dtype) if z is not None else None
        dbias = new((Di,), torch.float32) if dt_bias is not None else None
        ds0 = torch.empty_like(initial_state) if initial_state is not None else None
        if workspace is None:
            workspace = _scratch(need, x.device)
        st = load().ssm_scan_bwd(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z),
                                 _addr(dt_bias), _addr(initial_state), dy.data_ptr(), _addr(dfinal_state), dx.data_ptr(),
                                 ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _addr(dD), _addr(dz),
                                 _addr(dbias), _addr(ds0), _addr(cu_seqlens),
                                 _pitches(x, dt, B, C, x if z is None else z, dy), n_seq, rows, T, Di, N,
                                 GDN_DT_SOFTPLUS if softplus else 0, code, _addr(workspace), _room(workspace),
                                 _at(stream, x))
    if st:
        _raise("ssm_scan_bwd", st)
    return dx, ddt, dA, dB, dC, dD, dz, dbias, ds0


def ssm_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, slots=None, state_out=None, softplus=True, y=None,
             stream=None):
    """One token of ssm_scan_fwd for each row: x, dt, z [B,Di], B, C [B,N] (rows may
    lie apart) against a pool of states [slots,Di,N] fp32, updated in place unless
    state_out is given; slots int32 [B]: each row's page, -1 for an idle row (y =
    0).  Returns y [B,Di]."""
    if y is None and stream is None:
        r = (_front or _quick()).scan_step(x, dt, A, B, C, state, D, z, dt_bias, slots, state_out, softplus)
        if r is not NotImplemented:
            return r
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a [B,channels] CUDA tensor")
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise TypeError("A must be a [channels,N] CUDA tensor")
    rows, Di = x.shape
    code, N, dtype = _dtype_code(x), A.shape[1], x.dtype
    _dense(A, "A", (Di, N), torch.float32)
    steps = [_row(t, name, (rows, n), dtype) for t, name, n in
             ((x, "x", Di), (dt, "dt", Di), (B, "B", N), (C, "C", N), (x if z is None else z, "z", Di))]
    _maybe(D, "D", (Di,), torch.float32)
    _maybe(dt_bias, "dt_bias", (Di,), torch.float32)
    n = _pages(state, "state", (Di, N), torch.float32, slots, rows)
    if state_out is None:
        state_out = state
    elif state_out is not state:
        _dense(state_out, "state_out", state.shape, torch.float32)
        if state_out.data_ptr() != state.data_ptr():
            _apart(state_out, state, "state and state_out")
    _same_device(x, dt, A, B, C, state, D, z, dt_bias, slots, state_out, y)
    with _device(x, stream):
        if y is None:
            y = torch.empty(rows, Di, dtype=dtype, device=x.device)
        else:
            _dense(y, "y", (rows, Di), dtype)
            for t, name in ((x, "x"), (dt, "dt"), (B, "B"), (C, "C"), (z, "z"), (state, "state"), (state_out, "state_out")):
                _apart(y, t, f"{name} and y")
        st = load().ssm_step(x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D), _addr(z),
                             _addr(dt_bias), state.data_ptr(), state_out.data_ptr(), _addr(slots), y.data_ptr(),
                             (ctypes.c_longlong * 5)(*steps), rows, Di, N, n, GDN_DT_SOFTPLUS if softplus else 0, code,
                             _at(stream, x))
    if st:
        _raise("ssm_step", st)
    return y


def _gated(x, gate, weight, gate_first, sigmoid):
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise TypeError("x must be a [B,T,heads,D] CUDA tensor")
    code, D = _dtype_code(x), x.shape[3]
    _strided(x, "x", x.shape, x.dtype)
    _strided(gate, "gate", x.shape, x.dtype)
    shared = weight is None or weight.dim() == 1
    _maybe(weight, "weight", (D,) if shared else (x.shape[2], D), torch.float32)
    flags = (GDN_GATE_FIRST if gate_first else 0) | (GDN_GATE_SIGMOID if sigmoid else 0) | (GDN_W_SHARED if shared else 0)
    return code, flags


def gated_norm_fwd(x, gate, weight=None, eps=1e-6, gate_first=False, sigmoid=False, y=None, stream=None):
    """The root-mean-square norm of each head with its gate: weight n(x) act(gate),
    or weight n(x act(gate)) with gate_first; act is SiLU or the sigmoid.  x, gate
    [B,T,H,D] (last dimension contiguous; heads first, as the attention gives them,
    are x.transpose(1, 2)); weight [D] or [H,D] fp32.  Returns y [B,T,H,D],
    contiguous."""
    if y is None and stream is None:
        r = (_front or _quick()).gated(x, gate, weight, eps, gate_first, sigmoid)
        if r is not NotImplemented:
            return r
    code, flags = _gated(x, gate, weight, gate_first, sigmoid)
    _same_device(x, gate, weight, y)
    with _device(x, stream):
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _dense(y, "y", x.shape, x.dtype)
            _apart(y, x, "x and y")
            _apart(y, gate, "gate and y")
        st = load().gated_norm_fwd(x.data_ptr(), gate.data_ptr(), _addr(weight), y.data_ptr(), _pitches(x, gate), *x.shape,
                                   eps, flags, code, _at(stream, x))
    if st:
        _raise("gated_norm_fwd", st)
    return y


def gated_norm_bwd(dy, x, gate, weight=None, eps=1e-6, gate_first=False, sigmoid=False, workspace=None, stream=None):
    """Backward of gated_norm_fwd: (dx, dgate, dweight).  dx is dense, its dimensions
    in x's order; dgate is contiguous; dweight is fp32 in weight's shape ([D], the
    sum over the heads, without one)."""
    if workspace is None and stream is None:
        r = (_front or _quick()).gated_back(dy, x, gate, weight, eps, gate_first, sigmoid)
        if r is not NotImplemented:
            return r
    code, flags = _gated(x, gate, weight, gate_first, sigmoid)
    _strided(dy, "dy", x.shape, x.dtype)
    _same_device(x, dy, gate, weight, workspace)
    B, T, H, D = x.shape
    need = _bytes("gated_norm_bwd_workspace_bytes", B, T, H, D, flags)
    with _device(x, stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if _overlaps(x) else torch.empty_like(x)
        dgate = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty((D,) if flags & GDN_W_SHARED else (H, D), dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = _scratch(need, x.device)
        st = load().gated_norm_bwd(dy.data_ptr(), x.data_ptr(), gate.data_ptr(), _addr(weight), dx.data_ptr(),
                                   dgate.data_ptr(), dw.data_ptr(), _pitches(x, gate, dy, dx), B, T, H, D, eps, flags,
                                   code, _addr(workspace), _room(workspace), _at(stream, x))
    if st:
        _raise("gated_norm_bwd", st)
    return dx, dgate, dw


def _block(x, post_weight, scale, weight):
    """(rows, C, groups, code) of [...,C] rows; a scale [C] is one group's."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x must be a [...,C] CUDA tensor")
    C, code = x.shape[-1], _dtype_code(x)
    _dense(x, "x", x.shape, x.dtype)
    _maybe(post_weight, "post_weight", (C,), torch.float32)
    _maybe(weight, "weight", (C,), torch.float32)
    rows = x.numel() // C if C else 0
    groups = 0
    if scale is not None:
        if not isinstance(scale, torch.Tensor) or scale.dim() not in (1, 2):
            raise TypeError("scale must be a [C] or [groups,C] CUDA tensor")
        groups = 1 if scale.dim() == 1 else scale.shape[0]
        _dense(scale, "scale", (C,) if scale.dim() == 1 else (groups, C), torch.float32)
        if groups == 0 or rows % groups:
            raise ValueError(f"{groups} groups do not divide {rows} rows")
    return rows, C, groups, code


def block_norm_fwd(x, residual, post_weight=None, scale=None, weight=None, eps=1e-6, stream=None):
    """The norm after a block, its scale, the residual's sum and the norm before the
    next block: h = residual + scale n(x) post_weight, y = n(h) weight.  x, residual
    [...,C]; post_weight, weight [C] fp32; scale [C] or [groups,C] fp32, each group's
    for an equal run of rows.  Returns (y, h)."""
    if stream is None:
        r = (_front or _quick()).block(x, residual, post_weight, scale, weight, eps)
        if r is not NotImplemented:
            return r
    rows, C, groups, code = _block(x, post_weight, scale, weight)
    _dense(residual, "residual", x.shape, x.dtype)
    _same_device(x, residual, post_weight, scale, weight)
    with _device(x, stream):
        y, h = torch.empty_like(x), torch.empty_like(x)
        st = load().block_norm_fwd(x.data_ptr(), residual.data_ptr(), _addr(post_weight), _addr(scale), _addr(weight),
                                   y.data_ptr(), h.data_ptr(), rows, C, groups, eps, code, _at(stream, x))
    if st:
        _raise("block_norm_fwd", st)
    return y, h


def block_norm_bwd(dy, dh, x, h, post_weight=None, scale=None, weight=None, eps=1e-6, workspace=None, stream=None):
    """Backward of block_norm_fwd at the h that it returned.  dh (or None): the
    gradient that reaches h past the norm.  Returns (dx, dresidual, dpost_weight,
    dscale, dweight): the weights' in fp32, None for those that are not given."""
    if workspace is None and stream is None:
        r = (_front or _quick()).block_back(dy, dh, x, h, post_weight, scale, weight, eps)
        if r is not NotImplemented:
            return r
    rows, C, groups, code = _block(x, post_weight, scale, weight)
    _dense(dy, "dy", x.shape, x.dtype)
    _dense(h, "h", x.shape, x.dtype)
    _maybe(dh, "dh", x.shape, x.dtype)
    _same_device(x, dy, dh, h, post_weight, scale, weight, workspace)
    need = _bytes("block_norm_bwd_workspace_bytes", rows, C, groups)
    with _device(x, stream):
        dx, dres = torch.empty_like(x), torch.empty_like(x)
        dw1, ds, dw2 = (torch.empty_like(t) if t is not None else None for t in (post_weight, scale, weight))
        if workspace is None:
            workspace = _scratch(need, x.device)
        st = load().block_norm_bwd(dy.data_ptr(), _addr(dh), x.data_ptr(), h.data_ptr(), _addr(post_weight), _addr(scale),
                                   _addr(weight), dx.data_ptr(), dres.data_ptr(), _addr(dw1), _addr(ds), _addr(dw2), rows, C,
                                   groups, eps, code, _addr(workspace), _room(workspace), _at(stream, x))
    if st:
        _raise("block_norm_bwd", st)
    return dx, dres, dw1, ds, dw2


def device_error(stream=None) -> int:
    """Synchronise ``stream`` and read/clear the library's device error word."""
    return int(load().gdn_get_device_error(_stream(stream)))


def set_wait_limit(us: int) -> None:
    """Wall-clock limit in microseconds of each bounded device wait (0 = default)."""
    _raise("gdn_set_wait_limit", load().gdn_set_wait_limit(int(us)))


def set_cluster_shape(heads_per_cluster: int = 0, wy_ctas_per_cluster: int = 0) -> None:
    """Cluster shape of the tcgen05 path (0, 0: automatic)."""
    _raise("gdn_set_cluster_shape", load().gdn_set_cluster_shape(int(heads_per_cluster), int(wy_ctas_per_cluster)))


def launch_count() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().gdn_launch_count())


def status_string(code: int) -> str:
    return load().gdn_status_string(int(code)).decode()
