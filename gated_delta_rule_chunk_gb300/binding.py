"""Thin binding over libgdn (include/gdn.h, include/gdn_attn.h): argument marshalling only,
through ctypes (the attention calls: through a small compiled module).

Every step of the method runs in the CUDA kernels behind the C ABI. Torch is
used here only to own device memory (outputs, workspace) and to name the
current stream. If ``libgdn.so`` is missing the first call raises: there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import threading
from typing import Optional

import torch

from . import build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_FLAG_QK_L2NORM = 1
GDN_FLAG_BUILD_CHUNK_INDICES = 2
GDN_FLAG_CHANNEL_GATES = 4
GDN_FLAG_WORKSPACE_GUARDS = 8
GDN_NUM_STAGE_EVENTS = 5
DEV_STATUS_BITS = {1: "bad cu_seqlens", 2: "chunk overflow", 4: "bad chunk table",
                   8: "on-chip wait timed out", 16: "non-finite state or output",
                   32: "index out of range (GDN_DEBUG build)", 64: "bad page table",
                   128: "bad length or position"}
GDN_DEV_DEBUG_INDEX = 32

# Every entry point include/gdn.h and include/gdn_attn.h declare.
EXPORTED = ("gdn_check_desc", "gdn_nt_max", "gdn_workspace_size", "gdn_build_chunk_indices",
            "gdn_chunk_fwd", "gdn_read_status", "gdn_status_string", "gdn_chunk_fwd_noalloc",
            "gdn_noalloc_read_status", "gdn_test_scan_timeout", "gdn_workspace_regions",
            "gdn_debug_build", "gdn_test_debug_poison",
            "gdn_recurrent_fwd", "gdn_conv_front", "gdn_bwd_workspace_size", "gdn_chunk_bwd",
            "gdn_attn_check_desc", "gdn_attn_workspace_size", "gdn_attn_front",
            "gdn_attn_prefill", "gdn_attn_decode", "gdn_test_attn_prefix", "gdn_test_attn_tiles",
            "gdn_test_attn_timeout")
GDN_NOALLOC_SCRATCH_BYTES = 64 << 20
GDN_ATTN_ROPE_INTERLEAVED = 1


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = f"{what}: " if what else ""
        # (without loading the library: a missing one is reported from under load_library's lock)
        text = status_string(status) if _lib is not None else "library not loaded"
        super().__init__(f"{msg}libgdn status {status} ({text})")


class GdnDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32),
                ("Hv", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("chunk_size", ctypes.c_int32), ("nt_max", ctypes.c_int32),
                ("qkv_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("l2norm_eps", ctypes.c_float),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("stage_events", ctypes.c_void_p)]


class GdnAttnDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32),
                ("Hk", ctypes.c_int32), ("D", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("max_pos", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("norm_eps", ctypes.c_float),
                ("status", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libgdn.so (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise GdnError(-6, f"{path} is missing (build it with __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        vp, i32, P = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER
        lib.gdn_check_desc.argtypes = [P(GdnDesc)]
        lib.gdn_check_desc.restype = ctypes.c_int
        lib.gdn_nt_max.argtypes = [i32, i32, i32]
        lib.gdn_nt_max.restype = i32
        lib.gdn_workspace_size.argtypes = [P(GdnDesc)]
        lib.gdn_workspace_size.restype = ctypes.c_size_t
        lib.gdn_build_chunk_indices.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
        lib.gdn_build_chunk_indices.restype = ctypes.c_int
        lib.gdn_chunk_fwd.argtypes = [P(GdnDesc), vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                      vp, vp, vp, vp]
        lib.gdn_chunk_fwd.restype = ctypes.c_int
        lib.gdn_chunk_fwd_noalloc.argtypes = lib.gdn_chunk_fwd.argtypes
        lib.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.gdn_noalloc_read_status.argtypes = [vp, vp]
        lib.gdn_noalloc_read_status.restype = ctypes.c_int
        lib.gdn_debug_build.argtypes = []
        lib.gdn_debug_build.restype = ctypes.c_int
        lib.gdn_test_debug_poison.argtypes = [i32]
        lib.gdn_test_debug_poison.restype = None
        lib.gdn_test_scan_timeout.argtypes = [ctypes.c_uint32]
        lib.gdn_test_scan_timeout.restype = None
        lib.gdn_workspace_regions.argtypes = [P(GdnDesc), vp, vp, ctypes.c_int]
        lib.gdn_workspace_regions.restype = ctypes.c_int
        lib.gdn_recurrent_fwd.argtypes = [P(GdnDesc), vp, vp, vp, vp, vp, ctypes.c_float, vp,
                                          vp, vp, vp, vp]
        lib.gdn_recurrent_fwd.restype = ctypes.c_int
        lib.gdn_conv_front.argtypes = [P(GdnDesc), vp, vp, i32, vp, vp, vp, vp, vp, vp, vp,
                                       i32, vp]
        lib.gdn_conv_front.restype = ctypes.c_int
        lib.gdn_bwd_workspace_size.argtypes = [P(GdnDesc)]
        lib.gdn_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_chunk_bwd.argtypes = [P(GdnDesc), vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                      vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn_chunk_bwd.restype = ctypes.c_int
        lib.gdn_attn_check_desc.argtypes = [P(GdnAttnDesc)]
        lib.gdn_attn_check_desc.restype = ctypes.c_int
        lib.gdn_attn_workspace_size.argtypes = [P(GdnAttnDesc)]
        lib.gdn_attn_workspace_size.restype = ctypes.c_size_t
        lib.gdn_attn_front.argtypes = [P(GdnAttnDesc)] + [vp] * 13
        lib.gdn_attn_front.restype = ctypes.c_int
        lib.gdn_test_attn_prefix.argtypes = [i32]
        lib.gdn_test_attn_prefix.restype = None
        lib.gdn_test_attn_tiles.argtypes = [i32]
        lib.gdn_test_attn_tiles.restype = None
        lib.gdn_test_attn_timeout.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
        lib.gdn_test_attn_timeout.restype = None
        lib.gdn_attn_prefill.argtypes = [P(GdnAttnDesc), vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                         vp]
        lib.gdn_attn_prefill.restype = ctypes.c_int
        lib.gdn_attn_decode.argtypes = [P(GdnAttnDesc), vp, vp, vp, vp, vp, i32, ctypes.c_float,
                                        vp, vp, vp]
        lib.gdn_attn_decode.restype = ctypes.c_int
        lib.gdn_read_status.argtypes = [P(GdnDesc), vp, vp]
        lib.gdn_read_status.restype = ctypes.c_int
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return (_lib or load_library()).gdn_status_string(int(status)).decode()
    except Exception:
        return "unknown"


gdn_status_string = status_string


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return GDN_F32
    if dt == torch.bfloat16:
        return GDN_BF16
    raise TypeError(f"unsupported dtype {dt}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_desc(T: int, N: int, H: int, Hv: int, qkv_dtype: torch.dtype,
              out_dtype: Optional[torch.dtype] = None, nt_max: int = 0, flags: int = 0,
              l2norm_eps: float = 0.0, dk: int = 128, dv: int = 128) -> GdnDesc:
    return GdnDesc(T=T, N=N, H=H, Hv=Hv, dk=dk, dv=dv, chunk_size=64, nt_max=nt_max,
                   qkv_dtype=_dtype_code(qkv_dtype),
                   out_dtype=_dtype_code(out_dtype or qkv_dtype), flags=flags,
                   l2norm_eps=l2norm_eps, workspace=None, workspace_bytes=0, stage_events=None)


def gdn_check_desc(desc: GdnDesc) -> int:
    return load_library().gdn_check_desc(ctypes.byref(desc))


def gdn_nt_max(T: int, N: int, chunk_size: int = 64) -> int:
    return load_library().gdn_nt_max(T, N, chunk_size)


def gdn_workspace_size(desc: GdnDesc) -> int:
    return int(load_library().gdn_workspace_size(ctypes.byref(desc)))


def alloc_workspace(desc: GdnDesc, device) -> torch.Tensor:
    n = gdn_workspace_size(desc)
    if n == 0:
        raise GdnError(load_library().gdn_check_desc(ctypes.byref(desc)), "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def gdn_build_chunk_indices(cu_seqlens: Optional[torch.Tensor], T: int, nt_max: int,
                            N: Optional[int] = None, status: Optional[torch.Tensor] = None,
                            stream=None):
    """Build the [nt_max, 2] chunk table and [N+1] chunk offsets on the device."""
    dev = cu_seqlens.device if cu_seqlens is not None else torch.device("cuda")
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (N or 1)
    table = torch.empty(nt_max, 2, dtype=torch.int32, device=dev)
    offsets = torch.empty(N + 1, dtype=torch.int32, device=dev)
    rc = load_library().gdn_build_chunk_indices(_ptr(cu_seqlens), N, T, nt_max, _ptr(table),
                                                _ptr(offsets), _ptr(status),
                                                _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_build_chunk_indices")
    return table, offsets


def gdn_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, scale: Optional[float] = None,
                  initial_state: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None,
                  chunk_indices: Optional[torch.Tensor] = None,
                  output_final_state: bool = True, out_dtype: Optional[torch.dtype] = None,
                  use_qk_l2norm: bool = False, l2norm_eps: float = 0.0,
                  build_chunk_indices: bool = False, nt_max: int = 0,
                  out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None,
                  stage_events=None, return_desc: bool = False, extra_flags: int = 0):
    """Chunked gated-delta-rule forward through the C ABI.

    q, k [T, H, d]; v [T, Hv, d] with d = 128 or 64 (fp32 or bf16, CUDA,
    contiguous); beta fp32 [T, Hv]; g fp32 [T, Hv] (one gate per token) or
    [T, Hv, d] (one gate per key channel); initial_state fp32 [N, Hv, d, d] or
    None; cu_seqlens int32 [N + 1] or None. Returns (out [T, Hv, d], final_state
    or None).
    """
    T, H, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    flags = (GDN_FLAG_QK_L2NORM if use_qk_l2norm else 0) | (
        GDN_FLAG_BUILD_CHUNK_INDICES if build_chunk_indices else 0) | (
        GDN_FLAG_CHANNEL_GATES if g.dim() == 3 else 0) | extra_flags
    out_dtype = out_dtype or (out.dtype if out is not None else q.dtype)
    desc = make_desc(T, N, H, Hv, q.dtype, out_dtype, nt_max=nt_max, flags=flags,
                     l2norm_eps=l2norm_eps, dk=dk, dv=dv)
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if out is None:
        out = torch.empty(T, Hv, dv, dtype=out_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, Hv, dv, dk, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(desc, q.device)
    desc.workspace = workspace.data_ptr()
    desc.workspace_bytes = workspace.numel()
    ev_arr = None
    if stage_events is not None:
        ev_arr = (ctypes.c_void_p * GDN_NUM_STAGE_EVENTS)(*[int(e) for e in stage_events])
        desc.stage_events = ctypes.cast(ev_arr, ctypes.c_void_p)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    rc = load_library().gdn_chunk_fwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        _ptr(initial_state), _ptr(cu_seqlens), _ptr(chunk_indices), _ptr(out),
        _ptr(final_state), _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_chunk_fwd")
    if return_desc:
        return out, final_state, desc, workspace
    return out, final_state


def gdn_recurrent_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                      beta: torch.Tensor, scale: Optional[float] = None,
                      initial_state: Optional[torch.Tensor] = None,
                      cu_seqlens: Optional[torch.Tensor] = None,
                      output_final_state: bool = True, out_dtype: Optional[torch.dtype] = None,
                      use_qk_l2norm: bool = False, l2norm_eps: float = 0.0,
                      out: Optional[torch.Tensor] = None,
                      final_state: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None,
                      return_desc: bool = False):
    """Token-serial forward (decode / speculative verify) through the C ABI.

    Same tensors as gdn_chunk_fwd. `status`, if given, is a 256-byte-aligned
    device buffer of at least 4 bytes that receives the device status word
    (read it with gdn_read_status on the returned descriptor).
    Returns (out, final_state) or (out, final_state, desc).
    """
    T, H, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    out_dtype = out_dtype or (out.dtype if out is not None else q.dtype)
    desc = make_desc(T, N, H, Hv, q.dtype, out_dtype,
                     flags=GDN_FLAG_QK_L2NORM if use_qk_l2norm else 0,
                     l2norm_eps=l2norm_eps, dk=dk, dv=dv)
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if out is None:
        out = torch.empty(T, Hv, dv, dtype=out_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, Hv, dv, dk, dtype=torch.float32, device=q.device)
    if status is not None:
        desc.workspace = status.data_ptr()
        desc.workspace_bytes = status.numel() * status.element_size()
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    rc = load_library().gdn_recurrent_fwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state),
        _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_recurrent_fwd")
    if return_desc:
        return out, final_state, desc
    return out, final_state


def gdn_conv_front(x: torch.Tensor, conv_w: torch.Tensor, H: int, Hv: int,
                   conv_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, use_qk_l2norm: bool = False,
                   l2norm_eps: float = 0.0, output_state: bool = True,
                   conv_state_out: Optional[torch.Tensor] = None, n_snapshots: int = 0,
                   status: Optional[torch.Tensor] = None, stream=None,
                   return_desc: bool = False, q: Optional[torch.Tensor] = None,
                   k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """Front end through the C ABI: x [T, C] (C = 2*H*128 + Hv*128, bf16 or fp32),
    conv_w fp32 [C, d_conv], conv_state fp32 [N, C, d_conv - 1] or None.
    Returns (q, k, v, conv_state_out or None, snapshots or None[, desc])."""
    T, C = x.shape
    d_conv = conv_w.shape[1]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    desc = make_desc(T, N, H, Hv, x.dtype, x.dtype,
                     flags=GDN_FLAG_QK_L2NORM if use_qk_l2norm else 0, l2norm_eps=l2norm_eps)
    for name, t in (("x", x), ("conv_w", conv_w)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    q = torch.empty(T, H, 128, dtype=x.dtype, device=x.device) if q is None else q
    k = torch.empty(T, H, 128, dtype=x.dtype, device=x.device) if k is None else k
    v = torch.empty(T, Hv, 128, dtype=x.dtype, device=x.device) if v is None else v
    if conv_state_out is None and output_state:
        conv_state_out = torch.empty(N, C, d_conv - 1, dtype=torch.float32, device=x.device)
    snaps = (torch.empty(N, n_snapshots, C, d_conv - 1, dtype=torch.float32, device=x.device)
             if n_snapshots > 0 else None)
    if status is not None:
        desc.workspace = status.data_ptr()
        desc.workspace_bytes = status.numel() * status.element_size()
    rc = load_library().gdn_conv_front(
        ctypes.byref(desc), _ptr(x), _ptr(conv_w), int(d_conv), _ptr(conv_state),
        _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(conv_state_out), _ptr(snaps),
        int(n_snapshots), _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_conv_front")
    if return_desc:
        return q, k, v, conv_state_out, snaps, desc
    return q, k, v, conv_state_out, snaps


def gdn_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                  beta: torch.Tensor, d_out: torch.Tensor, scale: Optional[float] = None,
                  initial_state: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None,
                  d_final_state: Optional[torch.Tensor] = None,
                  chunk_indices: Optional[torch.Tensor] = None, nt_max: int = 0,
                  workspace: Optional[torch.Tensor] = None, stream=None,
                  return_desc: bool = False, grads: Optional[dict] = None,
                  stage_events=None):
    """Backward of gdn_chunk_fwd through the C ABI (scalar gates, no L2 norm).

    Same inputs as the forward call plus d_out [T, Hv, d] (fp32 or bf16) and
    d_final_state fp32 [N, Hv, d, d] or None. Returns a dict of fp32 gradients
    dq, dk [T, H, d], dv [T, Hv, d], dg, dbeta [T, Hv] and d_initial_state
    [N, Hv, d, d]."""
    T, H, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    desc = make_desc(T, N, H, Hv, q.dtype, d_out.dtype, nt_max=nt_max, dk=dk, dv=dv,
                     flags=GDN_FLAG_CHANNEL_GATES if g.dim() == 3 else 0)
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("d_out", d_out)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    dev = q.device
    f32 = torch.float32
    grads = grads if grads is not None else dict(dq=torch.zeros(T, H, dk, dtype=f32, device=dev),
                 dk=torch.zeros(T, H, dk, dtype=f32, device=dev),
                 dv=torch.zeros(T, Hv, dv, dtype=f32, device=dev),
                 dg=torch.zeros(T, Hv, dtype=f32, device=dev),
                 dbeta=torch.zeros(T, Hv, dtype=f32, device=dev),
                 d_initial_state=torch.empty(N, Hv, dv, dk, dtype=f32, device=dev))
    if workspace is None:
        n = int(load_library().gdn_bwd_workspace_size(ctypes.byref(desc)))
        if n == 0:
            raise GdnError(load_library().gdn_check_desc(ctypes.byref(desc)), "bwd workspace")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    desc.workspace = workspace.data_ptr()
    desc.workspace_bytes = workspace.numel()
    ev_arr = None
    if stage_events is not None:
        ev_arr = (ctypes.c_void_p * GDN_NUM_STAGE_EVENTS)(*[int(e) for e in stage_events])
        desc.stage_events = ctypes.cast(ev_arr, ctypes.c_void_p)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    rc = load_library().gdn_chunk_bwd(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        _ptr(initial_state), _ptr(cu_seqlens), _ptr(chunk_indices), _ptr(d_out),
        _ptr(d_final_state), _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]),
        _ptr(grads["dg"]), _ptr(grads["dbeta"]), _ptr(grads["d_initial_state"]),
        _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_chunk_bwd")
    if return_desc:
        return grads, desc, workspace
    return grads


def gdn_read_status(desc: GdnDesc, stream=None) -> int:
    """Copy the device status word of the last call on desc.workspace (synchronizes)."""
    host = torch.zeros(1, dtype=torch.int32).pin_memory()
    rc = load_library().gdn_read_status(ctypes.byref(desc), _ptr(host), _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_read_status")
    (torch.cuda.current_stream() if stream is None else stream).synchronize()
    return int(host.item())


def gdn_chunk_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                          beta: torch.Tensor, scale: Optional[float] = None,
                          initial_state: Optional[torch.Tensor] = None,
                          cu_seqlens: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None,
                          final_state: Optional[torch.Tensor] = None,
                          out_dtype: Optional[torch.dtype] = None, stream=None):
    """The forward pass through gdn_chunk_fwd_noalloc: the library's own static
    scratch replaces the workspace (for callers that cannot allocate device
    memory; here torch only provides the caller's inputs and outputs)."""
    T, H, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    out_dtype = out_dtype or (out.dtype if out is not None else q.dtype)
    desc = make_desc(T, N, H, Hv, q.dtype, out_dtype, dk=dk, dv=dv,
                     flags=GDN_FLAG_CHANNEL_GATES if g.dim() == 3 else 0)
    if out is None:
        out = torch.empty(T, Hv, dv, dtype=out_dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty(N, Hv, dv, dk, dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    rc = load_library().gdn_chunk_fwd_noalloc(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
        _ptr(initial_state), _ptr(cu_seqlens), None, _ptr(out), _ptr(final_state),
        _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_chunk_fwd_noalloc")
    return out, final_state


def gdn_noalloc_read_status(stream=None) -> int:
    """Device status word of the last gdn_chunk_fwd_noalloc call on the current device
    (it lives in the library's static scratch; synchronizes the stream)."""
    host = torch.zeros(1, dtype=torch.int32).pin_memory()
    rc = load_library().gdn_noalloc_read_status(_ptr(host), _stream_handle(stream))
    if rc != 0:
        raise GdnError(rc, "gdn_noalloc_read_status")
    (torch.cuda.current_stream() if stream is None else stream).synchronize()
    return int(host.item())


def gdn_test_scan_timeout(polls: int) -> None:
    """Testing hook: with polls > 0 the bf16 scan waits that many polls on an event that
    never happens and takes its timeout path (GDN_DEV_TIMEOUT); 0 turns it off."""
    load_library().gdn_test_scan_timeout(int(polls))


def gdn_debug_build() -> bool:
    """Whether the loaded library is the GDN_DEBUG build (device-side index checks)."""
    return bool(load_library().gdn_debug_build())


def gdn_test_debug_poison(on: bool) -> None:
    """Testing hook of the GDN_DEBUG build: aim one intra CTA's M copies one slot past the
    end of their region, which the device check must catch (GDN_DEV_DEBUG_INDEX)."""
    load_library().gdn_test_debug_poison(1 if on else 0)


def gdn_workspace_regions(desc: GdnDesc):
    """[(begin, end)] byte ranges of the workspace regions for this descriptor."""
    b = (ctypes.c_size_t * 16)()
    e = (ctypes.c_size_t * 16)()
    n = load_library().gdn_workspace_regions(ctypes.byref(desc), b, e, 16)
    if n < 0:
        raise GdnError(n, "gdn_workspace_regions")
    return [(int(b[i]), int(e[i])) for i in range(n)]


# ---------------------------------------------------------------- softmax attention
# A call with a `stream` of its own that allocates (outputs, workspace) takes the memory from the
# current stream's: it then comes after what the current stream holds, and is refused where only one
# of the two streams is being captured. With all of them given it waits for nothing.
_attn_module = None


def _attn():
    """The compiled marshalling of the attention calls (csrc/attn_torch.cpp), bound to the
    loaded library. Raises if it has not been built, or for another torch or Python."""
    global _attn_module
    lib = load_library()
    with _lock:
        if _attn_module is None:
            path, abi = build.MODULE, build.module_abi()
            if not os.path.exists(path):
                raise GdnError(-6, f"{path} is missing (build it with __graft_entry__.build())")
            if build.module_built_for() != abi:
                raise GdnError(-6, f"{path} was not built for {abi} (build it with "
                                   "__graft_entry__.build())")
            spec = importlib.util.spec_from_file_location("_attn_torch", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.init(GdnError, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.gdn_attn_front, lib.gdn_attn_prefill, lib.gdn_attn_decode,
                lib.gdn_attn_workspace_size, lib.gdn_attn_check_desc)))
            _attn_module = module
        return _attn_module


def make_attn_desc(T: int, N: int, H: int, Hk: int, D: int, in_dtype: torch.dtype = torch.bfloat16,
                   out_dtype: Optional[torch.dtype] = None, page_size: int = 0, n_pages: int = 0,
                   max_pages: int = 0, rot_dim: int = 0, max_pos: int = 0, flags: int = 0,
                   norm_eps: float = 0.0) -> GdnAttnDesc:
    return GdnAttnDesc(T, N, H, Hk, D, page_size, n_pages, max_pages, rot_dim, max_pos,
                       _dtype_code(in_dtype), _dtype_code(out_dtype or in_dtype), flags, norm_eps,
                       None, None, 0)


def gdn_attn_check_desc(desc: GdnAttnDesc) -> int:
    return load_library().gdn_attn_check_desc(ctypes.byref(desc))


def gdn_attn_workspace_size(desc: GdnAttnDesc) -> int:
    return int(load_library().gdn_attn_workspace_size(ctypes.byref(desc)))


def gdn_attn_front(x: torch.Tensor, H: int, Hk: int, D: int,
                   q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, norm_eps: float = 0.0,
                   rope: Optional[torch.Tensor] = None, interleaved: bool = False,
                   cu_seqlens: Optional[torch.Tensor] = None,
                   kv_lens: Optional[torch.Tensor] = None,
                   page_table: Optional[torch.Tensor] = None,
                   k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                   output_kv: bool = True, out_dtype: Optional[torch.dtype] = None,
                   q: Optional[torch.Tensor] = None, k: Optional[torch.Tensor] = None,
                   v: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                   stream=None):
    """Front end of an attention layer through the C ABI.

    x [T, (H + 2 Hk) * D] (fp32 or bf16), channels q | k | v. Per head of q and k: RMS norm
    with q_weight / k_weight (fp32 [D]; None leaves that norm out), then the rotation of the
    first rope.shape[1] elements by the rows of `rope` (fp32 [max_pos, rot], see
    rope.rope_table) at the token's position. With page_table [N, max_pages] int32, k_cache
    and v_cache [n_pages, Hk, page_size, D], k and v are appended to the cache; kv_lens [N]
    int32 are the cache's lengths after that (None: the tokens are the sequence's first).
    out_dtype (fp32 or bf16) defaults to the cache's, else to x's. Returns (q [T, H, D], k,
    v [T, Hk, D]), the last two None when output_kv is false; q, k, v may be given. `status`,
    if given, is one int32 on the device that receives the device status word.
    """
    return (_attn_module or _attn()).front(
        x, H, Hk, D, q_weight, k_weight, norm_eps, rope, interleaved, cu_seqlens, kv_lens,
        page_table, k_cache, v_cache, output_kv, out_dtype, q, k, v, status,
        None if stream is None else stream.cuda_stream)


def gdn_attn_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                     return_lse: bool = False, lse: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None):
    """Causal attention of packed prompts through the C ABI: q [T, H, D], k, v [T, Hk, D]
    bf16, D = 128 or 64, H a multiple of Hk; cu_seqlens int32 [N + 1] or None (one
    sequence). Returns out [T, H, D], or (out, lse) with lse fp32 [T, H] when return_lse."""
    return (_attn_module or _attn()).prefill(
        q, k, v, cu_seqlens, scale, out_dtype, out, return_lse, lse, status,
        None if stream is None else stream.cuda_stream)


def gdn_attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    page_table: torch.Tensor, kv_lens: torch.Tensor, shared_len: int = 0,
                    scale: Optional[float] = None, out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, return_lse: bool = False,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None):
    """Decode attention over the paged cache through the C ABI: q [N, H, D] (one token a
    sequence) or [N, n_q, H, D] bf16; k_cache, v_cache [n_pages, Hk, page_size, D] bf16;
    page_table int32 [N, max_pages]; kv_lens int32 [N], the call's tokens included. The first
    shared_len tokens (a multiple of page_size) are the same pages for every sequence and are
    read once for all. `workspace` (uint8, gdn_attn_workspace_size bytes) is allocated when
    not given. Returns out with q's shape, or (out, lse) when return_lse."""
    return (_attn_module or _attn()).decode(
        q, k_cache, v_cache, page_table, kv_lens, shared_len, scale, out_dtype, out, return_lse,
        lse, workspace, status, None if stream is None else stream.cuda_stream)


def gdn_test_attn_prefix(always: bool) -> None:
    """Testing hook: gdn_attn_decode gives a common prefix its own pass at every size."""
    load_library().gdn_test_attn_prefix(1 if always else 0)


def gdn_test_attn_tiles(tiles: int) -> None:
    """Testing hook: gdn_attn_prefill's work items hold 1 or 2 row tiles; 0: by its rule."""
    load_library().gdn_test_attn_tiles(tiles)


def gdn_test_attn_timeout(polls: int, item: int = 0) -> None:
    """Testing hook: with polls > 0 the tensor-core attention kernel waits that many polls, before
    a CTA's `item`-th work item, for an event that never happens (GDN_DEV_TIMEOUT); 0 turns it off."""
    load_library().gdn_test_attn_timeout(int(polls), int(item))
