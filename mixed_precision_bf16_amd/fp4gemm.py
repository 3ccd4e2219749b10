"""ctypes binding of ``libfp4gemm.so`` (argument marshalling only).

Every step of the GEMM runs in the HIP library; this module turns NumPy /
PyTorch buffers into pointers and status codes into exceptions.  PyTorch is
used for device memory and the current HIP stream.  There is no fallback: if
the library is missing or the device is not gfx950, calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import operator
import os
import re
import struct

import numpy as np

from . import build as _build

NVFP4 = 0
MXFP4 = 1
GROUP = {NVFP4: 16, MXFP4: 32}

_c_i64 = ctypes.c_int64
_c_vp = ctypes.c_void_p
_c_sz = ctypes.c_size_t


class _KVCacheDesc(ctypes.Structure):
    """fp4_kv_cache of include/fp4gemm.h."""
    _fields_ = [("data", _c_vp), ("pages", _c_i64), ("page_size", _c_i64), ("kv_heads", _c_i64),
                ("head_dim", _c_i64), ("format", ctypes.c_int32), ("k_alpha", ctypes.c_float),
                ("v_alpha", ctypes.c_float)]


class _AttentionArgs(ctypes.Structure):
    """fp4_attention_args of include/fp4gemm.h."""
    _fields_ = [("q", _c_vp), ("out", _c_vp), ("lse", _c_vp), ("page_table", _c_vp), ("seq_lens", _c_vp),
                ("q_offsets", _c_vp), ("sinks", _c_vp), ("batch", _c_i64), ("q_rows", _c_i64), ("q_heads", _c_i64),
                ("max_q", _c_i64), ("page_columns", _c_i64), ("page_stride", _c_i64), ("q_token_stride", _c_i64),
                ("q_head_stride", _c_i64), ("out_token_stride", _c_i64), ("out_head_stride", _c_i64),
                ("window", _c_i64), ("causal", ctypes.c_int32), ("act_type", ctypes.c_int32),
                ("scale", ctypes.c_float), ("workspace", _c_vp), ("workspace_bytes", _c_sz)]


# the same structure as bytes, which is quicker to fill
_PACK_ATTENTION = struct.Struct("@7Q11q2if4x2Q")


# name -> (restype, argtypes); mirrors include/fp4gemm.h
_SIGNATURES = {
    "fp4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fp4_repack_size": (ctypes.c_int, [_c_i64, _c_i64, ctypes.c_int, ctypes.POINTER(_c_sz), ctypes.POINTER(_c_sz)]),
    "fp4_repack": (ctypes.c_int, [_c_vp, _c_vp, _c_i64, _c_i64, ctypes.c_int, _c_vp, _c_vp]),
    "fp4_unpack": (ctypes.c_int, [_c_vp, _c_vp, _c_i64, _c_i64, ctypes.c_int, _c_vp, _c_vp]),
    "fp4_gemm_workspace_size": (ctypes.c_int, [_c_i64, _c_i64, _c_i64, ctypes.c_int, ctypes.POINTER(_c_sz)]),
    "fp4_gemm": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, ctypes.c_int, _c_vp, _c_sz,
                                _c_vp]),
    "fp4_gemm_noalloc": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, ctypes.c_int, _c_vp]),
    "fp4_gemm_noalloc_max_workspace": (ctypes.c_size_t, []),
    "fp4_gemm_f16": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, ctypes.c_int, _c_vp,
                                    _c_sz, _c_vp]),
    "fp4_dequant": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, ctypes.c_int, _c_vp]),
    "fp4_dequant_f16": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, ctypes.c_int, _c_vp]),
    "fp4_gemm_ex": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, ctypes.c_int, ctypes.c_int,
                                   ctypes.c_float, _c_vp, _c_sz, _c_vp]),
    "fp4_quantize": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_i64, ctypes.c_int, ctypes.c_float, _c_vp]),
    "fp4_native_repack_size": (ctypes.c_int, [_c_i64, _c_i64, ctypes.POINTER(_c_sz), ctypes.POINTER(_c_sz)]),
    "fp4_native_repack": (ctypes.c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "fp4_native_unpack": (ctypes.c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "fp4_gemm_native_workspace_size": (ctypes.c_int, [_c_i64, _c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
    "fp4_gemm_native": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, ctypes.c_float, _c_vp,
                                       _c_sz, _c_vp]),
    "fp4_moe_gemm": (ctypes.c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64,
                                    _c_i64, _c_i64, _c_i64, ctypes.c_int, _c_vp]),
    "fp4_kv_cache_size": (ctypes.c_int, [_c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_int, ctypes.POINTER(_c_sz)]),
    "fp4_kv_append": (ctypes.c_int, [ctypes.POINTER(_KVCacheDesc), _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64,
                                     _c_i64, _c_i64, ctypes.c_int, _c_vp]),
    "fp4_kv_read": (ctypes.c_int, [ctypes.POINTER(_KVCacheDesc), _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_i64,
                                   _c_i64, _c_i64, ctypes.c_int, _c_vp]),
    "fp4_attention_workspace_size": (ctypes.c_int, [ctypes.POINTER(_KVCacheDesc), _c_vp, ctypes.POINTER(_c_sz)]),
    "fp4_attention": (ctypes.c_int, [ctypes.POINTER(_KVCacheDesc), _c_vp, _c_vp]),
}

STATUS = {0: "FP4_OK", 1: "FP4_ERR_NULL", 2: "FP4_ERR_SHAPE", 3: "FP4_ERR_FORMAT", 4: "FP4_ERR_VALUE",
          5: "FP4_ERR_WORKSPACE", 6: "FP4_ERR_DEVICE", 7: "FP4_ERR_HIP"}


class Fp4Error(RuntimeError):
    """A library call returned a non-zero status."""

    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().fp4_status_string(status).decode()
        super().__init__(f"{what}: {STATUS.get(status, status)} ({msg})")


_LIB = None


def lib_path() -> str:
    return _build.LIB_PATH


def lib():
    """Load the library (building it once if it was never built)."""
    global _LIB
    if _LIB is None:
        path = _build.ensure_built()
        handle = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def header_functions():
    """Names of the functions declared in include/fp4gemm.h."""
    hdr = os.path.join(_build.ROOT, "include", "fp4gemm.h")
    text = open(hdr).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(fp4_\w+)\s*\(", text, re.M)))


def _check(status: int, what: str):
    if status != 0:
        raise Fp4Error(status, what)


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(_c_vp)


# ------------------------------------------------------------------ host API
def repack_size(N: int, K: int, fmt: int):
    wq, sq = _c_sz(), _c_sz()
    _check(lib().fp4_repack_size(N, K, fmt, ctypes.byref(wq), ctypes.byref(sq)), "fp4_repack_size")
    return wq.value, sq.value


def repack(codes: np.ndarray, scales: np.ndarray, N: int, K: int, fmt: int):
    """Canonical codes [N][K/2] and scales [N][K/G] (uint8, host) -> packed (wq, sq)."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.uint8)
    if codes.size != N * (K // 2) or scales.size != N * (K // GROUP.get(fmt, 1)):
        raise ValueError("codes / scales do not match N, K, format")
    nw, ns = repack_size(N, K, fmt)
    wq = np.empty(nw, dtype=np.uint8)
    sq = np.empty(ns, dtype=np.uint8)
    _check(lib().fp4_repack(_np_ptr(codes), _np_ptr(scales), N, K, fmt, _np_ptr(wq), _np_ptr(sq)), "fp4_repack")
    return wq, sq


def unpack(wq: np.ndarray, sq: np.ndarray, N: int, K: int, fmt: int):
    """Packed (wq, sq) -> canonical (codes [N][K/2], scales [N][K/G])."""
    nw, ns = repack_size(N, K, fmt)
    wq = np.ascontiguousarray(wq, dtype=np.uint8)
    sq = np.ascontiguousarray(sq, dtype=np.uint8)
    if wq.size != nw or sq.size != ns:
        raise ValueError("packed arrays have the wrong size")
    codes = np.empty((N, K // 2), dtype=np.uint8)
    scales = np.empty((N, K // GROUP[fmt]), dtype=np.uint8)
    _check(lib().fp4_unpack(_np_ptr(wq), _np_ptr(sq), N, K, fmt, _np_ptr(codes), _np_ptr(scales)), "fp4_unpack")
    return codes, scales


def workspace_size(m: int, N: int, K: int, fmt: int) -> int:
    b = _c_sz()
    _check(lib().fp4_gemm_workspace_size(m, N, K, fmt, ctypes.byref(b)), "fp4_gemm_workspace_size")
    return b.value


# ---------------------------------------------------------------- device API
def _dev_ptr(t):
    return _c_vp(t.data_ptr()) if t is not None else _c_vp(0)


def _on_device_of(ref, **tensors):
    """Raise ValueError unless every given tensor (None allowed) is a CUDA
    tensor on ref's device: a host pointer handed to a kernel would fault."""
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != ref.device):
            raise ValueError(f"{name} must be a CUDA tensor on {ref.device}")


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return _c_vp(stream.cuda_stream)


def new_workspace(m: int, N: int, K: int, fmt: int, device="cuda"):
    """A zero-filled workspace for fp4_gemm of this shape (None if none is needed)."""
    import torch
    nbytes = workspace_size(m, N, K, fmt)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def gemm(A, wq, sq, N: int, K: int, fmt: int, out=None, workspace=None, stream=None, alpha: float = 1.0):
    """Y = alpha * A . dequant(W)^T.  A: bfloat16 (fp4_gemm) or float16
    (fp4_gemm_f16) CUDA [m][K]; wq, sq: uint8 CUDA (packed).  alpha != 1 goes
    through fp4_gemm_ex.  Returns (or fills) a tensor [m][N] of A's dtype."""
    import torch
    if A.dtype not in (torch.bfloat16, torch.float16) or A.dim() != 2 or not A.is_cuda or not A.is_contiguous():
        raise ValueError("A must be a contiguous 2-D bfloat16 or float16 CUDA tensor")
    if A.shape[1] != K:
        raise ValueError("A must have K columns")
    for t in (wq, sq):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("wq / sq must be contiguous uint8 CUDA tensors")
    nw, ns = repack_size(N, K, fmt)
    if wq.numel() != nw or sq.numel() != ns:
        raise ValueError("packed weight tensors have the wrong size")
    m = A.shape[0]
    if out is None:
        out = torch.empty((m, N), dtype=A.dtype, device=A.device)
    elif out.shape != (m, N) or out.dtype != A.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor [m][N] of A's dtype")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    _on_device_of(A, wq=wq, sq=sq, out=out, workspace=workspace)
    wsb = workspace_size(m, N, K, fmt)
    if wsb and workspace is None:
        workspace = torch.zeros(wsb, dtype=torch.uint8, device=A.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if alpha != 1.0:
        act = 0 if A.dtype == torch.bfloat16 else 1
        _check(lib().fp4_gemm_ex(_dev_ptr(A), _dev_ptr(wq), _dev_ptr(sq), _dev_ptr(out), m, N, K, fmt, act, alpha,
                                 _dev_ptr(workspace), ws_bytes, _stream_handle(stream)), "fp4_gemm_ex")
        return out
    fn = lib().fp4_gemm if A.dtype == torch.bfloat16 else lib().fp4_gemm_f16
    _check(fn(_dev_ptr(A), _dev_ptr(wq), _dev_ptr(sq), _dev_ptr(out), m, N, K, fmt, _dev_ptr(workspace), ws_bytes,
              _stream_handle(stream)), "fp4_gemm")
    return out


def gemm_noalloc(A, wq, sq, N: int, K: int, fmt: int, out, stream=None):
    """fp4_gemm_noalloc: Y = A . dequant(W)^T with the library's own per-GPU
    scratch instead of a workspace (nothing is allocated; `out`, a contiguous
    bfloat16 CUDA tensor [m][N], must be given)."""
    import torch
    if A.dtype != torch.bfloat16 or A.dim() != 2 or not A.is_cuda or not A.is_contiguous() or A.shape[1] != K:
        raise ValueError("A must be a contiguous bfloat16 CUDA tensor [m][K]")
    for t in (wq, sq):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("wq / sq must be contiguous uint8 CUDA tensors")
    nw, ns = repack_size(N, K, fmt)
    if wq.numel() != nw or sq.numel() != ns:
        raise ValueError("packed weight tensors have the wrong size")
    m = A.shape[0]
    if out is None or out.shape != (m, N) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor [m][N]")
    _on_device_of(A, wq=wq, sq=sq, out=out)
    _check(lib().fp4_gemm_noalloc(_dev_ptr(A), _dev_ptr(wq), _dev_ptr(sq), _dev_ptr(out), m, N, K, fmt,
                                  _stream_handle(stream)), "fp4_gemm_noalloc")
    return out


def quantize(W, fmt: int, alpha: float = 1.0, stream=None):
    """fp4_quantize: BF16 CUDA weights [N][K] -> (codes uint8 [N][K/2], scales
    uint8 [N][K/G]) on the device, in the source order repack() takes."""
    import torch
    if W.dtype != torch.bfloat16 or W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D bfloat16 CUDA tensor")
    N, K = W.shape
    G = 16 if fmt == NVFP4 else 32
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((N, max(K // G, 1)), dtype=torch.uint8, device=W.device)
    _check(lib().fp4_quantize(_dev_ptr(W), _dev_ptr(codes), _dev_ptr(scales), N, K, fmt, alpha,
                              _stream_handle(stream)), "fp4_quantize")
    return codes, scales


def dequant(wq, sq, N: int, K: int, fmt: int, out=None, stream=None, dtype=None):
    """Weights [N][K] exactly as the GEMM feeds them to the matrix core:
    bfloat16 (default) or float16 (dtype=torch.float16)."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("dtype must be torch.bfloat16 or torch.float16")
    for t in (wq, sq):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("wq / sq must be contiguous uint8 CUDA tensors")
    nw, ns = repack_size(N, K, fmt)
    if wq.numel() != nw or sq.numel() != ns:
        raise ValueError("packed weight tensors have the wrong size")
    if out is None:
        out = torch.empty((N, K), dtype=dtype, device=wq.device)
    elif out.shape != (N, K) or out.dtype != dtype or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA tensor [N][K] of the requested dtype")
    _on_device_of(wq, sq=sq, out=out)
    fn = lib().fp4_dequant if dtype == torch.bfloat16 else lib().fp4_dequant_f16
    _check(fn(_dev_ptr(wq), _dev_ptr(sq), _dev_ptr(out), N, K, fmt, _stream_handle(stream)), "fp4_dequant")
    return out


def upload(wq: np.ndarray, sq: np.ndarray, device="cuda"):
    """Copy packed host arrays to device uint8 tensors."""
    import torch
    return (torch.from_numpy(np.ascontiguousarray(wq)).to(device),
            torch.from_numpy(np.ascontiguousarray(sq)).to(device))


def moe_gemm(A, wq, sq, sorted_ids, expert_offsets, N: int, K: int, fmt: int, E: int, a_div: int, out_rows: int,
             topk_weights=None, out=None, stream=None):
    """Grouped MoE GEMM (fp4_moe_gemm): for each expert e and assignment id in
    sorted_ids[expert_offsets[e]:expert_offsets[e+1]],
    out[id] = w[id] * A[id // a_div] . dequant(W_e)^T.  wq / sq hold the E
    experts' packed weights back to back (each repack_size(N, K, fmt)).  Rows
    of out not listed in sorted_ids are left as they were."""
    import torch
    if A.dtype != torch.bfloat16 or A.dim() != 2 or not A.is_cuda or not A.is_contiguous() or A.shape[1] != K:
        raise ValueError("A must be a contiguous bfloat16 CUDA tensor [a_rows][K]")
    nw, ns = repack_size(N, K, fmt)
    for t, n in ((wq, nw), (sq, ns)):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() != E * n:
            raise ValueError("wq / sq must be contiguous uint8 CUDA tensors holding E packed experts")
    for t, dt in ((sorted_ids, torch.int32), (expert_offsets, torch.int32)):
        if t.dtype != dt or not t.is_cuda or not t.is_contiguous() or t.dim() != 1:
            raise ValueError("sorted_ids / expert_offsets must be contiguous int32 CUDA vectors")
    if expert_offsets.numel() != E + 1:
        raise ValueError("expert_offsets must have E + 1 entries")
    if topk_weights is not None and (topk_weights.dtype != torch.float32 or not topk_weights.is_cuda
                                     or not topk_weights.is_contiguous() or topk_weights.numel() != out_rows):
        raise ValueError("topk_weights must be a contiguous float32 CUDA vector of out_rows entries")
    if out is None:
        out = torch.zeros((out_rows, N), dtype=torch.bfloat16, device=A.device)
    elif out.shape != (out_rows, N) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor [out_rows][N]")
    _on_device_of(A, wq=wq, sq=sq, sorted_ids=sorted_ids, expert_offsets=expert_offsets,
                  topk_weights=topk_weights, out=out)
    _check(lib().fp4_moe_gemm(_dev_ptr(A), _dev_ptr(wq), _dev_ptr(sq), _dev_ptr(sorted_ids), _dev_ptr(expert_offsets),
                              _dev_ptr(topk_weights), _dev_ptr(out), A.shape[0], a_div, out_rows,
                              sorted_ids.numel(), E, N, K, fmt, _stream_handle(stream)), "fp4_moe_gemm")
    return out


def native_repack(codes, scales, N: int, K: int):
    """fp4_native_repack: canonical MXFP4 codes / scales (host, uint8) -> native
    packed (wq, sq) as CPU uint8 tensors."""
    import numpy as np
    import torch
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.uint8)
    if codes.size != N * K // 2 or scales.size != N * (K // 32):
        raise ValueError("codes / scales have the wrong size")
    nw, ns = native_repack_size(N, K)
    wq = np.empty(nw, np.uint8)
    sq = np.empty(ns, np.uint8)
    _check(lib().fp4_native_repack(codes.ctypes.data_as(_c_vp), scales.ctypes.data_as(_c_vp), N, K,
                                   wq.ctypes.data_as(_c_vp), sq.ctypes.data_as(_c_vp)), "fp4_native_repack")
    return torch.from_numpy(wq), torch.from_numpy(sq)


def native_unpack(wq, sq, N: int, K: int):
    """Inverse of native_repack (host arrays or CPU tensors) -> (codes, scales) numpy."""
    import numpy as np
    wq = np.ascontiguousarray(wq.numpy() if hasattr(wq, "numpy") else wq, dtype=np.uint8)
    sq = np.ascontiguousarray(sq.numpy() if hasattr(sq, "numpy") else sq, dtype=np.uint8)
    codes = np.empty((N, K // 2), np.uint8)
    scales = np.empty((N, K // 32), np.uint8)
    _check(lib().fp4_native_unpack(wq.ctypes.data_as(_c_vp), sq.ctypes.data_as(_c_vp), N, K,
                                   codes.ctypes.data_as(_c_vp), scales.ctypes.data_as(_c_vp)), "fp4_native_unpack")
    return codes, scales


def native_workspace_size(m: int, N: int, K: int) -> int:
    b = _c_sz()
    _check(lib().fp4_gemm_native_workspace_size(m, N, K, ctypes.byref(b)), "fp4_gemm_native_workspace_size")
    return b.value


def native_repack_size(N: int, K: int):
    wqb, sqb = _c_sz(), _c_sz()
    _check(lib().fp4_native_repack_size(N, K, ctypes.byref(wqb), ctypes.byref(sqb)), "fp4_native_repack_size")
    return wqb.value, sqb.value


def gemm_native(A, wq, sq, N: int, K: int, out=None, workspace=None, stream=None, alpha: float = 1.0):
    """fp4_gemm_native: C = alpha * dequant(quantize_mxfp4(A)) . dequant(W)^T
    with W in the native layout; A bfloat16 CUDA [m][K]; wq / sq uint8 CUDA
    tensors of native_repack_size(N, K) bytes (upload native_repack's CPU
    tensors first)."""
    import torch
    if A.dtype != torch.bfloat16 or A.dim() != 2 or not A.is_cuda or not A.is_contiguous() or A.shape[1] != K:
        raise ValueError("A must be a contiguous bfloat16 CUDA tensor [m][K]")
    nw, ns = native_repack_size(N, K)
    for t, n in ((wq, nw), (sq, ns)):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
            raise ValueError("wq / sq must be contiguous uint8 CUDA tensors of native_repack_size(N, K) bytes")
    m = A.shape[0]
    if out is None:
        out = torch.empty((m, N), dtype=torch.bfloat16, device=A.device)
    elif out.shape != (m, N) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bfloat16 tensor [m][N]")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    _on_device_of(A, wq=wq, sq=sq, out=out, workspace=workspace)
    need = native_workspace_size(m, N, K)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().fp4_gemm_native(_dev_ptr(A), _dev_ptr(wq), _dev_ptr(sq), _dev_ptr(out), m, N, K, alpha,
                                 _dev_ptr(workspace), ws_bytes, _stream_handle(stream)), "fp4_gemm_native")
    return out


# ------------------------------------------------- FP4 key/value cache, attention
@functools.lru_cache(maxsize=256)
def kv_cache_size(pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: int) -> int:
    """Bytes of a cache of this shape (fp4_kv_cache_size)."""
    b = _c_sz()
    _check(lib().fp4_kv_cache_size(pages, page_size, kv_heads, head_dim, fmt, ctypes.byref(b)), "fp4_kv_cache_size")
    return b.value


class KVCache:
    """A paged FP4 key/value cache of one attention layer: `data` (a contiguous
    uint8 CUDA tensor of kv_cache_size bytes, in the layout that
    include/fp4gemm.h documents) and its shape.  k_alpha / v_alpha are the
    per-tensor scales of keys and values.  All are fixed once the object is
    made: the library's descriptor holds the data's address and the values."""

    __slots__ = ("_data", "_pages", "_page_size", "_kv_heads", "_head_dim", "_fmt", "_k_alpha", "_v_alpha", "_desc",
                 "_ref")

    data, pages, page_size, kv_heads, head_dim, fmt, k_alpha, v_alpha = (
        property(operator.attrgetter(name)) for name in __slots__[:8])

    def __init__(self, data, pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: int, k_alpha: float = 1.0,
                 v_alpha: float = 1.0):
        import torch
        if data.dtype != torch.uint8 or not data.is_cuda or not data.is_contiguous():
            raise ValueError("data must be a contiguous uint8 CUDA tensor")
        if data.numel() != kv_cache_size(pages, page_size, kv_heads, head_dim, fmt):
            raise ValueError("data does not have the cache's size")
        self._data, self._pages, self._page_size, self._kv_heads = data, pages, page_size, kv_heads
        self._head_dim, self._fmt, self._k_alpha, self._v_alpha = head_dim, fmt, k_alpha, v_alpha
        self._desc = _KVCacheDesc(data.data_ptr(), pages, page_size, kv_heads, head_dim, fmt, k_alpha, v_alpha)
        self._ref = ctypes.byref(self._desc)


def new_kv_cache(pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: int, k_alpha: float = 1.0,
                 v_alpha: float = 1.0, device="cuda") -> KVCache:
    """An uninitialized cache (slots may hold anything until they are appended to)."""
    import torch
    data = torch.empty(kv_cache_size(pages, page_size, kv_heads, head_dim, fmt), dtype=torch.uint8, device=device)
    return KVCache(data, pages, page_size, kv_heads, head_dim, fmt, k_alpha, v_alpha)


class _Guard:
    """Context of a call on another device than the current one, or on a given
    stream: the device is made current for the library call, and what the
    wrapper allocates belongs to the stream that the kernels run on."""

    __slots__ = ("handle", "_guards")

    def __init__(self, device, stream):
        import torch
        self._guards = [torch.cuda.device(device)]
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream must be a stream of {device}")
            self._guards.append(torch.cuda.stream(stream))
            self.handle = stream.cuda_stream
        else:
            self.handle = torch.cuda.current_stream(device).cuda_stream

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)


class _Current:
    """The same for the current stream of the current device: no state to set."""

    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return None


def _on_stream(device, stream):
    import torch
    if stream is None and torch._C._cuda_getDevice() == device.index:
        return _Current(torch._C._cuda_getCurrentRawStream(device.index))
    return _Guard(device, stream)


def _keep(device, stream, used, made=()):
    """After a launch on a given stream: the memory of the caller's tensors
    (`used`) is not handed out again before that stream has passed the launch,
    nor that of the tensors made on it (`made`) before the caller's stream has
    passed what it does with them until it drops them."""
    import torch
    for t in used:
        if t is not None:
            t.record_stream(stream)
    for t in made:
        t.record_stream(torch.cuda.current_stream(device))


def _act_type(dtype, what: str) -> int:
    import torch
    if dtype == torch.bfloat16:
        return 0
    if dtype == torch.float16:
        return 1
    raise ValueError(f"{what} must be bfloat16 or float16")


def _rows(t, what: str, tokens: int, heads: int, head_dim: int, device):
    """(token stride, head stride) of a [tokens][heads][head_dim] tensor."""
    if t.shape != (tokens, heads, head_dim) or t.device != device:
        raise ValueError(f"{what} must be a tensor [{tokens}][{heads}][{head_dim}] on {device}")
    a, b, c = t.stride()
    a, b = a if tokens > 1 else 0, b if heads > 1 else 0  # the stride of a single row means nothing
    if c != 1 or a % 8 or b % 8 or t.data_ptr() % 16:
        raise ValueError(f"{what} must have contiguous, 16-byte aligned rows")
    return a, b


def _vector(t, what: str, n: int, dtype, device):
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n} entries on {device}")
    return t.data_ptr()


def kv_append(cache: KVCache, k, v, slots, stream=None) -> None:
    """fp4_kv_append: quantize k, v (bfloat16 or float16 CUDA [tokens][kv_heads][head_dim],
    any token and head strides that are multiples of 8) into the cache at
    slots (int64 CUDA [tokens]; page * page_size + position in the page, a slot
    outside the cache is skipped, no slot twice)."""
    import torch
    act = _act_type(k.dtype, "k")
    dev = cache._data.device
    if v.dtype != k.dtype:
        raise ValueError("k and v must have the same type")
    n = k.shape[0]
    kt, kh = _rows(k, "k", n, cache._kv_heads, cache._head_dim, dev)
    vt, vh = _rows(v, "v", n, cache._kv_heads, cache._head_dim, dev)
    sp = _vector(slots, "slots", n, torch.int64, dev)
    with _on_stream(dev, stream) as s:
        st = lib().fp4_kv_append(cache._ref, k.data_ptr(), v.data_ptr(), sp, n, kt, kh, vt, vh, act, s)
    if st:
        _check(st, "fp4_kv_append")
    if stream is not None:
        _keep(dev, stream, (cache._data, k, v, slots))


def kv_read(cache: KVCache, slots, dtype=None, k_out=None, v_out=None, stream=None):
    """fp4_kv_read: the cache's rows at slots (int64 CUDA [tokens]) as
    (k, v), each [tokens][kv_heads][head_dim] of `dtype` (bfloat16 by default);
    zeros for a slot outside the cache.  k_out / v_out are filled if given."""
    import torch
    dev = cache._data.device
    given = [t.dtype for t in (k_out, v_out) if t is not None]
    if dtype is None:
        dtype = given[0] if given else torch.bfloat16
    act = _act_type(dtype, "dtype")
    if any(g != dtype for g in given):
        raise ValueError("k_out and v_out must have the requested type")
    n = slots.shape[0] if slots.dim() == 1 else -1
    sp = _vector(slots, "slots", n, torch.int64, dev)
    with _on_stream(dev, stream) as s:
        shape = (n, cache._kv_heads, cache._head_dim)
        kt = vt = cache._kv_heads * cache._head_dim  # strides of what is allocated here
        kh = vh = cache._head_dim
        made = []
        if k_out is None:
            made.append(k_out := torch.empty(shape, dtype=dtype, device=dev))
        else:
            kt, kh = _rows(k_out, "k_out", *shape, dev)
        if v_out is None:
            made.append(v_out := torch.empty(shape, dtype=dtype, device=dev))
        else:
            vt, vh = _rows(v_out, "v_out", *shape, dev)
        st = lib().fp4_kv_read(cache._ref, sp, n, k_out.data_ptr(), v_out.data_ptr(), kt, kh, vt, vh, act, s)
    if st:
        _check(st, "fp4_kv_read")
    if stream is not None:
        _keep(dev, stream, (cache._data, slots, k_out, v_out), made)
    return k_out, v_out


def _attention_shape(q, cache, page_table, seq_lens, q_offsets, max_q):
    """Checks of the tensors that every call has; (device, activation type,
    pointers, sizes, query strides) as fp4_attention_args takes them."""
    import torch
    dev = cache._data.device
    if q.dim() != 3:
        raise ValueError("q must be a tensor [q_rows][q_heads][head_dim]")
    act = _act_type(q.dtype, "q")
    rows, heads, _ = q.shape
    qt, qh = _rows(q, "q", rows, heads, cache._head_dim, dev)
    if (page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.device != dev
            or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError(f"page_table must be an int32 matrix [batch][columns] on {dev} with contiguous rows")
    batch, columns = page_table.shape
    offsets = 0
    if q_offsets is not None:
        offsets = _vector(q_offsets, "q_offsets", batch + 1, torch.int32, dev)
        if max_q is None:
            max_q = rows
    else:
        if batch and rows % batch:
            raise ValueError("q_rows must be a multiple of the batch without q_offsets")
        max_q = rows // batch if batch else 0
    pointers = page_table.data_ptr(), _vector(seq_lens, "seq_lens", batch, torch.int32, dev), offsets
    sizes = batch, rows, heads, max_q, columns, page_table.stride(0) if batch > 1 else columns
    return dev, act, pointers, sizes, (qt, qh)


def _pack_attention(*fields) -> bytes:
    try:
        return _PACK_ATTENTION.pack(*fields)
    except struct.error as e:
        raise ValueError(f"attention: {e}") from None


@functools.lru_cache(maxsize=1024)
def _attention_workspace(kv_heads, page_size, head_dim, fmt, batch, rows, heads, max_q, columns, offsets) -> int:
    c = _KVCacheDesc(None, 1, page_size, kv_heads, head_dim, fmt, 1.0, 1.0)
    a = _pack_attention(0, 0, 0, 0, 0, 4 if offsets else 0, 0, batch, rows, heads, max_q, columns, columns, 0, 0, 0, 0,
                        0, 1, 0, 1.0, 0, 0)
    b = _c_sz()
    _check(lib().fp4_attention_workspace_size(ctypes.byref(c), a, ctypes.byref(b)), "fp4_attention_workspace_size")
    return b.value


def attention_workspace_size(q, cache: KVCache, page_table, seq_lens, q_offsets=None, max_q=None) -> int:
    """Bytes of workspace that attention() needs for these shapes."""
    _, _, _, sizes, _ = _attention_shape(q, cache, page_table, seq_lens, q_offsets, max_q)
    return _attention_workspace(cache._kv_heads, cache._page_size, cache._head_dim, cache._fmt, *sizes[:5],
                                q_offsets is not None)


def attention(q, cache: KVCache, page_table, seq_lens, q_offsets=None, max_q=None, causal: bool = True,
              window: int = 0, scale=None, sinks=None, out=None, lse=None, return_lse: bool = False, workspace=None,
              stream=None):
    """fp4_attention: softmax(scale * q . K^T) . V over the cache.

    q: bfloat16 or float16 CUDA [q_rows][q_heads][head_dim]; page_table: int32
    [batch][columns], its rows at least `columns` apart, or one row for all
    (expand); seq_lens: int32 [batch], keys of each sequence, the query tokens'
    own among them.  The query rows of sequence b are q_offsets[b] ..
    q_offsets[b + 1] - 1 (int32 [batch + 1], never decreasing) or, without
    q_offsets, q_rows / batch each; they are its last positions.  max_q: about
    the most query tokens of a sequence, for the choice of kernel (default with
    q_offsets: q_rows; give it where the sequences are short: single tokens of 64
    sequences of 4000 keys take 227 us without it and 60 us with it).  window >
    0: only the last `window` positions up to the query's own.  scale:
    head_dim ** -0.5 by default.  sinks: float32 [q_heads].
    Returns out ([q_rows][q_heads][head_dim] of q's type) or (out, lse) with
    lse float32 [q_rows][q_heads]; rows that q_offsets gives to no sequence are
    not written (in what the wrapper allocates they hold anything)."""
    import torch
    dev, act, pointers, sizes, strides = _attention_shape(q, cache, page_table, seq_lens, q_offsets, max_q)
    rows, heads, dim = q.shape
    sink = _vector(sinks, "sinks", heads, torch.float32, dev) if sinks is not None else 0
    with _on_stream(dev, stream) as s:
        made = []
        if out is None:
            out = torch.empty_like(q) if q.is_contiguous() else torch.empty((rows, heads, dim), dtype=q.dtype, device=dev)
            made.append(out)
            ot, oh = heads * dim, dim
        elif out.dtype != q.dtype:
            raise ValueError("out must have q's type")
        else:
            ot, oh = _rows(out, "out", rows, heads, dim, dev)
        if lse is not None:
            if lse.dtype != torch.float32 or lse.shape != (rows, heads) or lse.device != dev or not lse.is_contiguous():
                raise ValueError(f"lse must be a contiguous float32 tensor [{rows}][{heads}] on {dev}")
        elif return_lse:
            made.append(lse := torch.empty((rows, heads), dtype=torch.float32, device=dev))
        if workspace is None:
            need = _attention_workspace(cache._kv_heads, cache._page_size, dim, cache._fmt, *sizes[:5],
                                        q_offsets is not None)
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        args = _pack_attention(q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else 0, *pointers, sink,
                               *sizes, *strides, ot, oh, window, 1 if causal else 0, act,
                               dim ** -0.5 if scale is None else scale, workspace.data_ptr(),
                               workspace.numel() * workspace.element_size())
        st = lib().fp4_attention(cache._ref, args, s)
    if st:
        _check(st, "fp4_attention")
    if stream is not None:
        _keep(dev, stream, (q, cache._data, page_table, seq_lens, q_offsets, sinks, out, lse, workspace), made)
    return (out, lse) if return_lse else out
