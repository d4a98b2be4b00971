"""Binding of libgdn.so (include/gdn.h). Argument marshalling only: by ctypes, and compiled
(csrc/binding_ext.cpp) for the calls that a decoding step makes in every layer.

Every step of the computation runs in the library's CUDA kernels; PyTorch only
allocates device memory and supplies the current CUDA stream. There is no CPU
or framework fallback: if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
from typing import Dict, NamedTuple, Optional, Tuple

import torch

from . import build as _build

GDN_OK = 0
GDN_ERR_INVALID_ARG = 1
GDN_ERR_UNSUPPORTED = 2
GDN_ERR_SHAPE = 3
GDN_ERR_CUDA = 4
GDN_ERR_INTERNAL = 5
GDN_ERR_SCRATCH_LIMIT = 6
GDN_NOALLOC_SCRATCH_BYTES = 32 << 20
GDN_F32 = 0
GDN_BF16 = 1
GDN_FLAG_PAIRWISE_WITHIN_BLOCK = 1
GDN_FLAG_QK_L2NORM = 2
GDN_FLAG_CHUNK128 = 4
GDN_FLAG_ROPE_PAIRS = 16
GDN_FLAG_GATE_SIGMOID = 32
GDN_FLAG_CONV_SILU = 64
GDN_FLAG_DT_SOFTPLUS = 128
GDN_FLAG_ZERO_PADDING = 256
GDN_CHUNK = 64
GDN_CHUNK128 = 128

# every symbol include/gdn.h declares
EXPORTED = ("gdn_chunk_residual_bytes", "gdn_chunk_bwd_workspace_bytes", "gdn_chunk_fwd",
            "gdn_chunk_bwd", "gdn_recurrent", "gdn_check_device_error", "gdn_status_string",
            "gdn_version", "gdn_profile_enable", "gdn_profile_read", "gdn_kernel_name",
            "gdn_chunk_fwd_noalloc", "gdn_replay_buffer_bytes", "gdn_replay_decode",
            "gdn_replay_state", "gdn_selftest_wait_timeout", "gdn_kv_append",
            "gdn_paged_attn_workspace_bytes", "gdn_paged_attn", "gdn_block_norm_fwd",
            "gdn_block_norm_workspace_bytes", "gdn_block_norm_bwd", "gdn_causal_conv_fwd",
            "gdn_causal_conv_workspace_bytes", "gdn_causal_conv_bwd", "gdn_selective_scan_residual_bytes",
            "gdn_selective_scan_workspace_bytes", "gdn_selective_scan_fwd",
            "gdn_selective_scan_bwd_workspace_bytes", "gdn_selective_scan_bwd", "gdn_page_plan")
KERNEL_COUNT = 40
GDN_REPLAY_MAX_TOKENS = 8


class GdnDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("Dk", ctypes.c_int), ("Dv", ctypes.c_int), ("g_per_channel", ctypes.c_int),
                ("dtype", ctypes.c_int), ("flags", ctypes.c_int)]


_ll, _vp = ctypes.c_longlong, ctypes.c_void_p


class GdnPagedDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("N", "B", "Hq", "Hk", "D", "page_size", "num_pages", "max_pages",
                                            "dtype", "flags")]


class GdnPagedCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_page_stride", _ll), ("k_head_stride", _ll), ("k_row_stride", _ll),
                ("v_page_stride", _ll), ("v_head_stride", _ll), ("v_row_stride", _ll), ("page_table", _vp),
                ("page_table_stride", _ll), ("cu_seqlens", _vp), ("kv_lens", _vp)]


class GdnTokens(ctypes.Structure):
    _fields_ = [("p", _vp), ("token_stride", _ll), ("head_stride", _ll)]


class GdnNormDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int), ("G", ctypes.c_int), ("C", ctypes.c_int), ("dtype", ctypes.c_int),
                ("flags", ctypes.c_int), ("eps", ctypes.c_float)]


class GdnRows(ctypes.Structure):
    _fields_ = [("p", _vp), ("row_stride", _ll), ("group_stride", _ll)]


class GdnNormParts(ctypes.Structure):
    _fields_ = [("x", GdnRows), ("gate", GdnRows), ("residual", GdnRows), ("w_post", _vp), ("res_scale", _vp),
                ("w_pre", _vp)]


class GdnNormGrads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dx", "dgate", "dresidual", "dw_post", "dres_scale", "dw_pre")]


class GdnPacked(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("B", ctypes.c_int), ("pool", ctypes.c_int), ("cu_seqlens", _vp), ("kv_lens", _vp),
                ("slots", _vp)]


class GdnConvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("C", "taps", "dtype", "flags")]


class GdnScanDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("D", "G", "S", "dtype", "flags")]


class GdnScanParts(ctypes.Structure):
    _fields_ = [(n, GdnRows) for n in ("u", "dt", "z", "B", "C")] + [(n, _vp) for n in ("A", "skip", "dt_bias", "h0")]


class GdnScanGrads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("du", "ddt", "dz", "dB", "dC", "dA", "dskip", "ddt_bias", "dh0")]


class GdnPlanDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "page_size", "max_pages", "num_free", "max_tokens")]


class GdnPlanOut(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("cu_seqlens", "kv_lens", "free_count", "requests", "positions", "slots")]


class GdnError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


_lock = threading.Lock()
_lib = None
_ext = None


def load(build_if_needed: bool = True) -> ctypes.CDLL:
    """Load libgdn.so (building it first when missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_needed and _build.lib_is_stale():
                _build.build_lib()
            if not os.path.exists(_build.LIB_PATH):
                raise RuntimeError(f"libgdn.so not found at {_build.LIB_PATH}; run the package build first")
            lib = ctypes.CDLL(_build.LIB_PATH)
            vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
            pd = ctypes.POINTER(GdnDims)
            lib.gdn_chunk_residual_bytes.argtypes = [pd]
            lib.gdn_chunk_residual_bytes.restype = sz
            lib.gdn_chunk_bwd_workspace_bytes.argtypes = [pd]
            lib.gdn_chunk_bwd_workspace_bytes.restype = sz
            lib.gdn_chunk_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp]
            lib.gdn_chunk_fwd.restype = i
            lib.gdn_chunk_bwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp]
            lib.gdn_chunk_bwd.restype = i
            lib.gdn_recurrent.argtypes = [pd, vp, vp, vp, vp, vp, vp, f, vp, vp, vp]
            lib.gdn_recurrent.restype = i
            lib.gdn_check_device_error.argtypes = []
            lib.gdn_check_device_error.restype = i
            lib.gdn_status_string.argtypes = [i]
            lib.gdn_status_string.restype = ctypes.c_char_p
            lib.gdn_version.argtypes = []
            lib.gdn_version.restype = i
            lib.gdn_profile_enable.argtypes = [i]
            lib.gdn_profile_enable.restype = i
            lib.gdn_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i), i]
            lib.gdn_profile_read.restype = i
            lib.gdn_kernel_name.argtypes = [i]
            lib.gdn_kernel_name.restype = ctypes.c_char_p
            lib.gdn_chunk_fwd_noalloc.argtypes = [pd, vp, vp, vp, vp, vp, vp, f, vp, vp, vp]
            lib.gdn_chunk_fwd_noalloc.restype = i
            lib.gdn_replay_buffer_bytes.argtypes = [pd, i]
            lib.gdn_replay_buffer_bytes.restype = sz
            lib.gdn_replay_decode.argtypes = [pd, i, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp]
            lib.gdn_replay_decode.restype = i
            lib.gdn_replay_state.argtypes = [pd, i, vp, vp, vp, vp, vp]
            lib.gdn_replay_state.restype = i
            lib.gdn_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp, vp]
            lib.gdn_selftest_wait_timeout.restype = i
            pp, pc, pt = (ctypes.POINTER(c) for c in (GdnPagedDims, GdnPagedCache, GdnTokens))
            lib.gdn_kv_append.argtypes = [pp, pc, pt, pt, pt, pt, vp, vp, i, i, vp]
            lib.gdn_kv_append.restype = i
            lib.gdn_paged_attn_workspace_bytes.argtypes = [pp, i, i]
            lib.gdn_paged_attn_workspace_bytes.restype = sz
            lib.gdn_paged_attn.argtypes = [pp, pc, pt, f, i, i, pt, vp, vp, vp]
            lib.gdn_paged_attn.restype = i
            pn, pr = ctypes.POINTER(GdnNormDims), ctypes.POINTER(GdnRows)
            pa, pg = ctypes.POINTER(GdnNormParts), ctypes.POINTER(GdnNormGrads)
            lib.gdn_block_norm_fwd.argtypes = [pn, pa, vp, vp, vp, vp]
            lib.gdn_block_norm_fwd.restype = i
            lib.gdn_block_norm_workspace_bytes.argtypes = [pn]
            lib.gdn_block_norm_workspace_bytes.restype = sz
            lib.gdn_block_norm_bwd.argtypes = [pn, pa, vp, pr, pr, pg, vp, vp]
            lib.gdn_block_norm_bwd.restype = i
            pq, pv, ps, pi = (ctypes.POINTER(c) for c in (GdnPacked, GdnConvDims, GdnScanDims, GdnScanParts))
            lib.gdn_causal_conv_fwd.argtypes = [pv, pq, pr, vp, vp, vp, i, pr, vp, vp]
            lib.gdn_causal_conv_fwd.restype = i
            lib.gdn_causal_conv_workspace_bytes.argtypes = [pv, pq]
            lib.gdn_causal_conv_workspace_bytes.restype = sz
            lib.gdn_causal_conv_bwd.argtypes = [pv, pq, pr, vp, vp, vp, pr, vp, vp, vp, vp, vp, vp, vp]
            lib.gdn_causal_conv_bwd.restype = i
            lib.gdn_selective_scan_residual_bytes.argtypes = [ps, pq]
            lib.gdn_selective_scan_residual_bytes.restype = sz
            lib.gdn_selective_scan_workspace_bytes.argtypes = [ps, pq, i]
            lib.gdn_selective_scan_workspace_bytes.restype = sz
            lib.gdn_selective_scan_fwd.argtypes = [ps, pq, pi, i, pr, vp, vp, vp, vp]
            lib.gdn_selective_scan_fwd.restype = i
            lib.gdn_selective_scan_bwd_workspace_bytes.argtypes = [ps, pq, i]
            lib.gdn_selective_scan_bwd_workspace_bytes.restype = sz
            lib.gdn_selective_scan_bwd.argtypes = [ps, pq, pi, vp, i, pr, vp, ctypes.POINTER(GdnScanGrads), vp, vp]
            lib.gdn_selective_scan_bwd.restype = i
            lib.gdn_page_plan.argtypes = [ctypes.POINTER(GdnPlanDims), vp, _ll, vp, vp, vp, vp,
                                          ctypes.POINTER(GdnPlanOut), vp]
            lib.gdn_page_plan.restype = i
            _lib = lib
    return _lib


def _compiled():
    """The compiled argument marshalling of the paged cache, block norm, convolution, scan and plan calls
    (csrc/binding_ext.cpp), built first when missing or stale."""
    global _ext
    load()
    with _lock:
        if _ext is None:
            if _build.ext_is_stale():
                _build.build_ext()
            spec = importlib.util.spec_from_file_location("_gdn_ext", _build.EXT_PATH)
            ext = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(ext)
            ext.set_error(GdnError)
            _ext = ext
    return _ext


def lib_path() -> str:
    return _build.LIB_PATH


def status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != GDN_OK:
        raise GdnError(fn, status, status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return GDN_F32
    if dt == torch.bfloat16:
        return GDN_BF16
    raise GdnError("dtype", GDN_ERR_UNSUPPORTED, f"unsupported dtype {dt} (float32 or bfloat16)")


def make_dims(q: torch.Tensor, v: torch.Tensor, g: torch.Tensor, flags: int = 0) -> GdnDims:
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    return GdnDims(B, T, H, Dk, Dv, int(g.dim() == 4), _dtype_code(q.dtype), int(flags))


def _stream(dev: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _require(tensors: Dict[str, Optional[torch.Tensor]], device: torch.device):
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda or t.device != device:
            raise GdnError(name, GDN_ERR_INVALID_ARG, f"{name} must be a CUDA tensor on {device}")
        if not t.is_contiguous():
            raise GdnError(name, GDN_ERR_INVALID_ARG, f"{name} must be contiguous")


def gdn_chunk_residual_bytes(dims: GdnDims) -> int:
    return int(load().gdn_chunk_residual_bytes(ctypes.byref(dims)))


def gdn_chunk_bwd_workspace_bytes(dims: GdnDims) -> int:
    return int(load().gdn_chunk_bwd_workspace_bytes(ctypes.byref(dims)))


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, scale: Optional[float] = None, *, out=None,
                  h_final=None, residuals=None, flags: int = 0):
    """Chunked forward. Returns (out [B,T,H,Dv], h_final fp32 [B,H,Dk,Dv], residuals)."""
    dev = q.device
    _require(dict(q=q, k=k, v=v, g=g, beta=beta, h0=h0, out=out, h_final=h_final,
                  residuals=residuals), dev)
    dims = make_dims(q, v, g, flags)
    if scale is None:
        scale = dims.Dk ** -0.5
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    if h_final is None:
        h_final = torch.empty((dims.B, dims.H, dims.Dk, dims.Dv), dtype=torch.float32, device=dev)
    if residuals is None:
        residuals = torch.empty(max(gdn_chunk_residual_bytes(dims), 1), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = load().gdn_chunk_fwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(h0), float(scale), _ptr(out), _ptr(h_final), _ptr(residuals),
                                  _stream(dev))
    _check("gdn_chunk_fwd", st)
    return out, h_final, residuals


def gdn_chunk_fwd_noalloc(q, k, v, g, beta, h0=None, scale: Optional[float] = None, *, out,
                          h_final, flags: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunked forward through the entry point that allocates nothing: the caller
    passes the outputs, the library keeps the residual records in its static
    device array (calls sharing it must not overlap on the GPU)."""
    dev = q.device
    _require(dict(q=q, k=k, v=v, g=g, beta=beta, h0=h0, out=out, h_final=h_final), dev)
    dims = make_dims(q, v, g, flags)
    if scale is None:
        scale = dims.Dk ** -0.5
    with torch.cuda.device(dev):
        st = load().gdn_chunk_fwd_noalloc(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                          _ptr(beta), _ptr(h0), float(scale), _ptr(out), _ptr(h_final),
                                          _stream(dev))
    _check("gdn_chunk_fwd_noalloc", st)
    return out, h_final


def gdn_chunk_bwd(q, k, v, g, beta, h0, residuals, dout, dh_final=None,
                  scale: Optional[float] = None, *, workspace=None, flags: int = 0,
                  need_dh0: bool = True, grads: Optional[Dict[str, torch.Tensor]] = None
                  ) -> Dict[str, torch.Tensor]:
    """Chunked backward (bf16 or fp32, the forward's dtype). Returns dq, dk, dv, dg, dbeta
    (input dtype) and dh0 (fp32).
    ``grads`` may supply preallocated output tensors under those names."""
    dev = q.device
    dims = make_dims(q, v, g, flags)
    if scale is None:
        scale = dims.Dk ** -0.5
    if grads is None:
        grads = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
                 "dg": torch.empty_like(g), "dbeta": torch.empty_like(beta)}
        grads["dh0"] = (torch.empty((dims.B, dims.H, dims.Dk, dims.Dv), dtype=torch.float32,
                                    device=dev) if need_dh0 else None)
    _require(dict(q=q, k=k, v=v, g=g, beta=beta, h0=h0, residuals=residuals, dout=dout,
                  dh_final=dh_final, workspace=workspace, **grads), dev)
    if workspace is None:
        workspace = torch.empty(max(gdn_chunk_bwd_workspace_bytes(dims), 1), dtype=torch.uint8,
                                device=dev)
    with torch.cuda.device(dev):
        st = load().gdn_chunk_bwd(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(h0), float(scale), _ptr(residuals), _ptr(dout),
                                  _ptr(dh_final), _ptr(grads["dq"]), _ptr(grads["dk"]),
                                  _ptr(grads["dv"]), _ptr(grads["dg"]), _ptr(grads["dbeta"]),
                                  _ptr(grads["dh0"]), _ptr(workspace), _stream(dev))
    _check("gdn_chunk_bwd", st)
    return grads


def gdn_recurrent(q, k, v, g, beta, h0=None, scale: Optional[float] = None, *, out=None,
                  h_final=None, flags: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Token-recurrent prefill / decode. h_final may be h0 (in-place carry)."""
    dev = q.device
    _require(dict(q=q, k=k, v=v, g=g, beta=beta, h0=h0, out=out, h_final=h_final), dev)
    dims = make_dims(q, v, g, flags)
    if scale is None:
        scale = dims.Dk ** -0.5
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    if h_final is None:
        h_final = torch.empty((dims.B, dims.H, dims.Dk, dims.Dv), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = load().gdn_recurrent(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(h0), float(scale), _ptr(out), _ptr(h_final), _stream(dev))
    _check("gdn_recurrent", st)
    return out, h_final


def gdn_replay_buffer_bytes(dims: GdnDims, L: int) -> int:
    return int(load().gdn_replay_buffer_bytes(ctypes.byref(dims), int(L)))


def replay_init(h0: torch.Tensor, L: int):
    """(ckpt, buffer, fill) for replay decode starting from state h0 [B,H,Dk,Dv] fp32:
    the checkpoint is a copy of h0, the buffer is empty (fill = 0)."""
    B, H, Dk, Dv = h0.shape
    dims = GdnDims(B, 1, H, Dk, Dv, 1, GDN_F32, 0)
    nbytes = gdn_replay_buffer_bytes(dims, L)
    if nbytes == 0 and B * H > 0:
        raise GdnError("gdn_replay_buffer_bytes", GDN_ERR_INVALID_ARG, f"bad dims or L={L}")
    ckpt = h0.detach().to(torch.float32).contiguous().clone()
    buffer = torch.empty(max(nbytes // 4, 4), dtype=torch.float32, device=h0.device)
    fill = torch.zeros((B, H), dtype=torch.int32, device=h0.device)
    return ckpt, buffer, fill


def gdn_replay_decode(q, k, v, g, beta, ckpt, buffer, fill, L: int, scale: Optional[float] = None, *,
                      out=None, flags: int = 0) -> torch.Tensor:
    """One decode step (T = 1) against checkpoint + buffer; advances fill, folds the
    buffer into ckpt when it is full. Returns out [B,1,H,Dv]."""
    dev = q.device
    _require(dict(q=q, k=k, v=v, g=g, beta=beta, ckpt=ckpt, buffer=buffer, fill=fill, out=out), dev)
    dims = make_dims(q, v, g, flags)
    if scale is None:
        scale = dims.Dk ** -0.5
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    with torch.cuda.device(dev):
        st = load().gdn_replay_decode(ctypes.byref(dims), int(L), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                      _ptr(beta), float(scale), _ptr(ckpt), _ptr(buffer), _ptr(fill),
                                      _ptr(out), _stream(dev))
    _check("gdn_replay_decode", st)
    return out


def gdn_replay_state(ckpt, buffer, fill, L: int, *, h_out=None) -> torch.Tensor:
    """The full state [B,H,Dk,Dv] fp32 that checkpoint + buffer stand for."""
    dev = ckpt.device
    _require(dict(ckpt=ckpt, buffer=buffer, fill=fill, h_out=h_out), dev)
    B, H, Dk, Dv = ckpt.shape
    dims = GdnDims(B, 1, H, Dk, Dv, 1, GDN_F32, 0)
    if h_out is None:
        h_out = torch.empty_like(ckpt)
    with torch.cuda.device(dev):
        st = load().gdn_replay_state(ctypes.byref(dims), int(L), _ptr(ckpt), _ptr(buffer), _ptr(fill),
                                     _ptr(h_out), _stream(dev))
    _check("gdn_replay_state", st)
    return h_out


def make_paged_dims(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor, flags: int = 0) -> GdnPagedDims:
    """dims of a paged call from q [N, Hq, D], k_cache [pages, Hk, page size, D] and page_table [B, pages]."""
    pages, Hk, page_size, D = k_cache.shape
    return GdnPagedDims(q.shape[0], page_table.shape[0], q.shape[1], Hk, D, page_size, pages, page_table.shape[1],
                        _dtype_code(k_cache.dtype), int(flags))


def make_norm_dims(x: torch.Tensor, eps: float = 1e-6, flags: int = 0) -> GdnNormDims:
    """dims of a block norm call from x [rows, C] or [rows..., groups, C]."""
    C, G = x.shape[-1], (1 if x.dim() == 2 else x.shape[-2])
    return GdnNormDims(x.numel() // max(C * G, 1), max(G, 1), C, _dtype_code(x.dtype), int(flags), float(eps))


def gdn_kv_append(k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, *, q=None, q_out=None, cos=None,
                  sin=None, flags: int = 0) -> Optional[torch.Tensor]:
    """Store packed new tokens' k, v [N, Hk, D] in the paged cache [pages, Hk, page size, D], in place;
    with cos, sin (fp32 [positions, rot / 2]) k is rotated by its position, and so is q [N, Hq, D].
    kv_lens counts the new tokens. Returns the rotated q (q_out, which may be q), or None without q.
    Serving only: with gradients enabled, tensors that require them are refused."""
    return (_ext or _compiled()).kv_append(k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, q, q_out, cos,
                                           sin, flags)


def gdn_paged_attn_workspace_bytes(dims: GdnPagedDims, max_q: int, max_kv: int) -> int:
    return int(load().gdn_paged_attn_workspace_bytes(ctypes.byref(dims), int(max_q), int(max_kv)))


def gdn_paged_attn(q, k_cache, v_cache, page_table, cu_seqlens, kv_lens, scale: Optional[float] = None, *,
                   max_q: Optional[int] = None, max_kv: Optional[int] = None, out=None, lse=None,
                   workspace=None) -> torch.Tensor:
    """Causal attention of the packed new tokens q [N, Hq, D] over the paged cache their keys were
    appended to. max_q, max_kv: the caller's bounds on new tokens and length of one sequence (they
    choose the kernel and its split; without them the largest possible are taken, which sends short
    decoding calls to the kernel of chunks: give max_q=1 there). lse: optional fp32
    [N, Hq] output, the log of each row's softmax sum. Returns out [N, Hq, D]. Serving only: with
    gradients enabled, tensors that require them are refused."""
    return (_ext or _compiled()).paged_attn(q, k_cache, v_cache, page_table, cu_seqlens, kv_lens, scale, max_q,
                                            max_kv, out, lse, workspace)


def gdn_block_norm_fwd(x, *, gate=None, residual=None, w_post=None, res_scale=None, w_pre=None, eps: float = 1e-6,
                       flags: int = 0):
    """h = residual + res_scale * (norm(x) * w_post * act(gate)) and y = norm(h) * w_pre, every part
    optional; the norm is over the last dimension. Returns (h, y or None, stats)."""
    return (_ext or _compiled()).block_norm_fwd(x, gate, residual, w_post, res_scale, w_pre, eps, flags)


def gdn_block_norm_workspace_bytes(dims: GdnNormDims) -> int:
    return int(load().gdn_block_norm_workspace_bytes(ctypes.byref(dims)))


def gdn_block_norm_bwd(x, stats, dh, dy=None, *, gate=None, residual=None, w_post=None, res_scale=None, w_pre=None,
                       eps: float = 1e-6, flags: int = 0, workspace=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of gdn_block_norm_fwd from dh (or None) and dy (with w_pre): dx, dgate, dresidual,
    dw_post, dres_scale, dw_pre in the inputs' dtype, None for absent parts."""
    grads = (_ext or _compiled()).block_norm_bwd(x, stats, dh, dy, gate, residual, w_post, res_scale, w_pre, eps,
                                                 flags, workspace)
    return dict(zip(("dx", "dgate", "dresidual", "dw_post", "dres_scale", "dw_pre"), grads))


def gdn_causal_conv_fwd(x, weight, bias=None, *, state0=None, state_final=None, slots=None, cu_seqlens=None,
                        kv_lens=None, max_q: Optional[int] = None, flags: int = 0, out=None):
    """Short causal convolution of every channel along the tokens (2 to 4 taps, weight [C, taps]), with silu by
    GDN_FLAG_CONV_SILU. x is [B, T, C], or packed [N, C] with cu_seqlens [B + 1]; states are the last taps - 1 inputs,
    [B, taps - 1, C], or rows `slots` [B] of pools (state_final may be state0: in place; a negative slot
    has no state). With kv_lens (cached tokens with the new ones) a sequence without earlier tokens starts from
    zeros. max_q: the caller's bound on one sequence's new tokens. Returns (y, state_final). Packed rows before
    the first sequence and behind the last are zeros, or in a given `out` left as they were; `out` shares no
    memory with the inputs. For gradients: causal_conv."""
    return (_ext or _compiled()).causal_conv_fwd(x, weight, bias, state0, state_final, slots, cu_seqlens, kv_lens, max_q,
                                                 flags, out)


def gdn_causal_conv_bwd(x, weight, bias, dy, *, state0=None, dstate=None, cu_seqlens=None, flags: int = 0,
                        workspace=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of gdn_causal_conv_fwd from dy and dstate (of the final states, or None): dx, dweight, dbias (with
    a bias) and dstate0 (with state0)."""
    grads = (_ext or _compiled()).causal_conv_bwd(x, weight, bias, dy, state0, dstate, cu_seqlens, flags, workspace)
    return dict(zip(("dx", "dweight", "dbias", "dstate0"), grads))


def gdn_selective_scan_fwd(u, dt, A, B, C, *, D=None, z=None, dt_bias=None, h0=None, h_final=None, slots=None,
                           cu_seqlens=None, kv_lens=None, max_q: Optional[int] = None, flags: int = 0, save: bool = False,
                           out=None, workspace=None):
    """Selective state space scan: h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t, y_t = (C_t . h_t + D u_t) silu(z_t),
    delta = dt + dt_bias or, with GDN_FLAG_DT_SOFTPLUS, its softplus. u, dt, z are [B, T, D], or packed [N, D] with
    cu_seqlens; B, C [..., groups, S] (S 8, 16, 32 or 64); A [D, S], D and dt_bias [D] and the states [B, D, S] float32,
    16-byte aligned. States, slots, kv_lens and max_q as in gdn_causal_conv_fwd; `out` may be u, dt or z itself.
    Returns (y, h_final, residuals): the residuals (with save) are the backward's. For gradients: selective_scan."""
    return (_ext or _compiled()).selective_scan_fwd(u, dt, A, B, C, D, z, dt_bias, h0, h_final, slots, cu_seqlens, kv_lens,
                                                    max_q, flags, save, out, workspace)


def gdn_selective_scan_bwd(u, dt, A, B, C, dy, residuals, *, D=None, z=None, dt_bias=None, dh_final=None,
                           need_dh0: bool = False, cu_seqlens=None, max_q: Optional[int] = None, flags: int = 0,
                           workspace=None) -> Dict[str, Optional[torch.Tensor]]:
    """Gradients of gdn_selective_scan_fwd from dy and dh_final (or None): du, ddt, dA, dB, dC, dD, dz, ddt_bias and,
    with need_dh0, dh0; None for absent parts."""
    grads = (_ext or _compiled()).selective_scan_bwd(u, dt, A, B, C, D, z, dt_bias, dy, residuals, dh_final, need_dh0,
                                                     cu_seqlens, max_q, flags, workspace)
    return dict(zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"), grads))


class PagePlan(NamedTuple):
    """What gdn_page_plan returns, all on the device and in one allocation: a part that is kept keeps all (clone it where
    max_tokens is large)."""

    cu_seqlens: torch.Tensor  # [B + 1] packed offsets of the granted new tokens
    kv_lens: torch.Tensor  # [B] cached tokens after the step
    free_count: torch.Tensor  # [1] pages left on the free list
    requests: torch.Tensor  # [max_tokens] request of each packed row, -1 behind the last
    positions: torch.Tensor  # [max_tokens] its position in the request
    slots: torch.Tensor  # [max_tokens] int64: its place in the cache, page * page_size + row


def gdn_page_plan(page_table, kv_lens, new_tokens, free_pages, free_count, *, page_size: int, max_tokens: int) -> PagePlan:
    """Plan a serving step from kv_lens [B] and new_tokens [B] (negative: tokens given back): pages are pushed
    on and popped off the stack free_pages[:free_count], page_table and free_pages change in place, and requests that
    do not fit the free pages or max_tokens, counted with all that is asked for before them, have no tokens in the
    step. The results feed gdn_kv_append, gdn_paged_attn, gdn_causal_conv_fwd and gdn_selective_scan_fwd; nothing is
    read back to the host."""
    return tuple.__new__(PagePlan, (_ext or _compiled()).page_plan(page_table, kv_lens, new_tokens, free_pages, free_count,
                                                                   page_size, max_tokens))


def gdn_selftest_wait_timeout(max_tries: int = 1024, device: Optional[torch.device] = None,
                              cycles: Optional[torch.Tensor] = None) -> None:
    """Launch the library's wait-timeout self-test kernel (see include/gdn.h). cycles: an
    optional int64 device tensor of three elements for the kernel's cycle counts."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    if cycles is not None:
        assert cycles.dtype == torch.int64 and cycles.numel() >= 3 and cycles.is_contiguous()
    with torch.cuda.device(dev):
        st = load().gdn_selftest_wait_timeout(int(max_tries), _ptr(cycles), _stream(dev))
    _check("gdn_selftest_wait_timeout", st)


def gdn_check_device_error() -> int:
    return int(load().gdn_check_device_error())


def gdn_version() -> int:
    return int(load().gdn_version())


def gdn_profile_enable(on: bool = True) -> None:
    _check("gdn_profile_enable", load().gdn_profile_enable(int(bool(on))))


def gdn_profile_read() -> Dict[str, Tuple[float, int]]:
    """{kernel name: (summed ms, launches)} since the last enable/read (kernels launched at least once)."""
    ms = (ctypes.c_double * KERNEL_COUNT)()
    n = (ctypes.c_int * KERNEL_COUNT)()
    _check("gdn_profile_read", load().gdn_profile_read(ms, n, KERNEL_COUNT))
    lib = load()
    return {lib.gdn_kernel_name(i).decode(): (float(ms[i]), int(n[i])) for i in range(KERNEL_COUNT) if n[i]}


def gdn_kernel_name(i: int) -> str:
    return load().gdn_kernel_name(int(i)).decode()


class GatedDeltaRule(torch.autograd.Function):
    """Chunked gated delta rule with the library's backward (bf16 or fp32)."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, scale, flags):
        out, h_final, res = gdn_chunk_fwd(q, k, v, g, beta, h0, scale, flags=flags)
        ctx.save_for_backward(q, k, v, g, beta, h0, res)
        ctx.scale = scale
        ctx.flags = flags
        return out, h_final

    @staticmethod
    def backward(ctx, dout, dh_final):
        q, k, v, g, beta, h0, res = ctx.saved_tensors
        grads = gdn_chunk_bwd(q, k, v, g, beta, h0, res, dout.contiguous(),
                              None if dh_final is None else dh_final.contiguous(), ctx.scale,
                              flags=ctx.flags, need_dh0=h0 is not None)
        return (grads["dq"], grads["dk"], grads["dv"], grads["dg"], grads["dbeta"],
                grads["dh0"] if h0 is not None else None, None, None)


def gated_delta_rule(q, k, v, g, beta, h0=None, scale: Optional[float] = None, flags: int = 0):
    """(out, h_final) of the chunked gated delta rule, differentiable through autograd."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return GatedDeltaRule.apply(q, k, v, g, beta, h0, float(scale), int(flags))


class BlockNorm(torch.autograd.Function):
    """gdn_block_norm_fwd with the library's backward."""

    @staticmethod
    def forward(ctx, x, gate, residual, w_post, res_scale, w_pre, eps, flags):
        h, y, stats = gdn_block_norm_fwd(x, gate=gate, residual=residual, w_post=w_post, res_scale=res_scale,
                                         w_pre=w_pre, eps=eps, flags=flags)
        # the residual's values are read only where the norm before the next block is
        ctx.save_for_backward(x, gate, residual if w_pre is not None else None, w_post, res_scale, w_pre, stats)
        ctx.eps, ctx.flags, ctx.has_residual = eps, flags, residual is not None
        ctx.set_materialize_grads(False)  # an unused output's gradient is None, not zeros to be read
        return h, y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dy):
        if dh is None and dy is None:
            return (None,) * 8
        x, gate, residual, w_post, res_scale, w_pre, stats = ctx.saved_tensors
        # without dy the norm before the next block is left out: dh passes it by, its weight gets zeros
        g = gdn_block_norm_bwd(x, stats, None if dh is None else dh.contiguous(),
                               None if dy is None else dy.contiguous(), gate=gate, residual=residual, w_post=w_post,
                               res_scale=res_scale, w_pre=None if dy is None else w_pre, eps=ctx.eps, flags=ctx.flags)
        dw_pre = torch.zeros_like(w_pre) if dy is None and w_pre is not None else g["dw_pre"]
        dresidual = dh if residual is None and ctx.has_residual else g["dresidual"]
        return g["dx"], g["dgate"], dresidual, g["dw_post"], g["dres_scale"], dw_pre, None, None


def block_norm(x, *, gate=None, residual=None, w_post=None, res_scale=None, w_pre=None, eps: float = 1e-6,
               flags: int = 0):
    """(h, y) of gdn_block_norm_fwd, differentiable once through autograd (y is None without w_pre)."""
    return BlockNorm.apply(x, gate, residual, w_post, res_scale, w_pre, float(eps), int(flags))


class CausalConv(torch.autograd.Function):
    """gdn_causal_conv_fwd with the library's backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, state0, cu_seqlens, max_q, flags):
        y, state = gdn_causal_conv_fwd(x, weight, bias, state0=state0, cu_seqlens=cu_seqlens, max_q=max_q, flags=flags)
        ctx.save_for_backward(x, weight, bias, state0, cu_seqlens)
        ctx.flags = flags
        ctx.set_materialize_grads(False)
        return y, state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dstate):
        if dy is None and dstate is None:
            return (None,) * 7
        x, weight, bias, state0, cu_seqlens = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else dy.contiguous()
        g = gdn_causal_conv_bwd(x, weight, bias, dy, state0=state0, dstate=None if dstate is None else dstate.contiguous(),
                                cu_seqlens=cu_seqlens, flags=ctx.flags)
        return g["dx"], g["dweight"], g["dbias"], g["dstate0"], None, None, None


def causal_conv(x, weight, bias=None, state0=None, *, cu_seqlens=None, max_q: Optional[int] = None, flags: int = 0):
    """(y, state_final) of gdn_causal_conv_fwd, differentiable once through autograd."""
    return CausalConv.apply(x, weight, bias, state0, cu_seqlens, max_q, int(flags))


class SelectiveScan(torch.autograd.Function):
    """gdn_selective_scan_fwd with the library's backward."""

    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, max_q, flags):
        y, h, kept = gdn_selective_scan_fwd(u, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, h0=h0, cu_seqlens=cu_seqlens,
                                            max_q=max_q, flags=flags, save=any(ctx.needs_input_grad))
        ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, kept)
        ctx.max_q, ctx.flags = max_q, flags
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh):
        if dy is None and dh is None:
            return (None,) * 12
        u, dt, A, B, C, D, z, dt_bias, cu_seqlens, kept = ctx.saved_tensors
        dy = torch.zeros_like(u) if dy is None else dy.contiguous()
        if dh is not None:
            dh = dh.contiguous()
            if dh.data_ptr() % 16:  # a part of a larger gradient: of a concatenation, say
                dh = dh.clone()
        g = gdn_selective_scan_bwd(u, dt, A, B, C, dy, kept, D=D, z=z, dt_bias=dt_bias, dh_final=dh, need_dh0=ctx.needs_input_grad[8],
                                   cu_seqlens=cu_seqlens, max_q=ctx.max_q, flags=ctx.flags)
        return (g["du"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddt_bias"], g["dh0"], None, None, None)


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, cu_seqlens=None,
                   max_q: Optional[int] = None, flags: int = 0):
    """(y, h_final) of gdn_selective_scan_fwd, differentiable once through autograd. Without gradients (torch.no_grad(),
    torch.inference_mode()) nothing is kept for a backward."""
    if not torch.is_grad_enabled():  # needs_input_grad asks the inputs alone
        return gdn_selective_scan_fwd(u, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, h0=h0, cu_seqlens=cu_seqlens, max_q=max_q,
                                      flags=int(flags))[:2]
    return SelectiveScan.apply(u, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, max_q, int(flags))
