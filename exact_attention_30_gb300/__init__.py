"""exact_attention_30_gb300 -- fused exact attention for GB300 (sm_103a).

A thin Python binding over the C ABI in ``include/fa.h`` (``libfa_gb300.so``).
It only marshals arguments: checks that tensors live on the GPU, are
contiguous and of the right dtype, allocates outputs with PyTorch (device
memory is PyTorch's job here) and passes raw pointers plus the current CUDA
stream to the library. Every step of the computation runs in the library's
CUDA kernels; there is no CPU path. If the shared library has not been built
(``python -m exact_attention_30_gb300.build``), every call raises.

    o, lse = fa_fwd(q, k, v, scale)                 # q,k,v: [B,H,N,d] cuda
    dq, dk, dv = fa_bwd(q, k, v, o, do, lse, scale)
    o, lse = fa_decode(q_new, k_cache, v_cache, scale)   # q_new: [B,H,Nq<=16,d]
    o, lse = fa_fwd(q, k, v, causal=True)            # causal self-attention
    o, lse = fa_fwd_varlen(q, k, v, cu_seqlens, max_seqlen)   # packed [total,H,d]

Serving from a paged cache (k_pages, v_pages: [pages, Hkv, page_size, d]):

    cos, sin = fa_rope_tables(max_positions, rot_dim, device="cuda")
    q = fa_kv_append(k, v, k_pages, v_pages, block_tables, seq_lens, cu_seqlens, q=q, cos=cos, sin=sin)
    o, lse = fa_decode_paged(q, k_pages, v_pages, block_tables, seq_lens)       # q: [B,Hq,Nq,d]
    o, lse = fa_decode_shared(q, k_pages, v_pages, prefix_pages, prefix_len, block_tables, seq_lens)
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct
import threading

import torch

__all__ = [
    "fa_fwd", "fa_bwd", "fa_bwd_stage", "fa_bwd_plan", "fa_fwd_varlen", "fa_bwd_varlen",
    "fa_bwd_varlen_workspace_bytes", "FA_CAUSAL", "fa_bwd_workspace_bytes", "fa_softmax_rows", "fa_decode",
    "fa_decode_workspace_bytes", "fa_decode_plan", "fa_check_device_status",
    "fa_rope_tables", "fa_kv_append", "fa_decode_paged", "fa_decode_paged_workspace_bytes",
    "fa_decode_shared", "fa_decode_shared_workspace_bytes", "fa_decode_shared_plan",
    "fa_debug_timeout_probe", "fa_status_string", "fa_version", "library_path", "load_library",
    "FA_OK", "FA_ERR_INVALID_ARG", "FA_ERR_UNSUPPORTED", "FA_ERR_CUDA", "FA_ERR_TIMEOUT",
    "FA_F32", "FA_BF16", "FAError", "FA_BWD_PREPROCESS", "FA_BWD_MAIN", "FA_BWD_DQ_CONVERT",
]

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_F32, FA_BF16 = 0, 1
FA_BWD_PREPROCESS, FA_BWD_MAIN, FA_BWD_DQ_CONVERT = 0, 1, 2
FA_CAUSAL = 1
FA_ROPE_INTERLEAVED = 2
_STAGE_FLAGS = {FA_BWD_PREPROCESS: 1 << 8, FA_BWD_MAIN: 2 << 8, FA_BWD_DQ_CONVERT: 4 << 8}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")
_lib = None

_vp, _ci, _cf, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong


# fa_paged_kv of include/fa.h and the three strides of a [B, H, N, d] view. They
# are passed as the packed bytes: for a decode step of one short sequence, what
# the host does per call is most of the time, and a ctypes structure costs more.
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_pack_pool = struct.Struct("@PPiiii6q").pack
_pack_strides = struct.Struct("@3q").pack

_SIGNATURES = {
    "fa_fwd": (_ci, [_vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _cf, _ci, _vp]),
    "fa_fwd_ex": (_ci, [_vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _cf, _ci, _ci, _vp]),
    "fa_fwd_varlen": (_ci, [_vp] * 6 + [_ci, _ci, _ci, _ci, _ci, _cf, _ci, _ci, _vp]),
    "fa_fwd_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci]),
    "fa_fwd_ws": (_ci, [_vp] * 6 + [_sz, _ci, _ci, _ci, _ci, _cf, _ci, _ci, _vp]),
    "fa_fwd_plan": (_ci, [_ci] * 7 + [ctypes.POINTER(_ci)] * 3),
    "fa_bwd_ex": (_ci, [_vp] * 10 + [_sz, _ci, _ci, _ci, _ci, _cf, _ci, _ci, _vp]),
    "fa_bwd_varlen_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci]),
    "fa_bwd_varlen": (_ci, [_vp] * 11 + [_sz, _ci, _ci, _ci, _ci, _ci, _cf, _ci, _ci, _vp]),
    "fa_bwd_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci]),
    "fa_bwd_plan": (_ci, [_ci] * 7 + [ctypes.POINTER(_ci)] * 3),
    "fa_bwd": (_ci, [_vp] * 10 + [_sz, _ci, _ci, _ci, _ci, _cf, _ci, _vp]),
    "fa_bwd_stage": (_ci, [_ci] + [_vp] * 10 + [_sz, _ci, _ci, _ci, _ci, _cf, _ci, _vp]),
    "fa_bwd_noalloc": (_ci, [_vp] * 9 + [_ci, _ci, _ci, _ci, _cf, _ci, _vp]),
    "fa_softmax_rows": (_ci, [_vp, _vp, _ci, _ci, _cf, _ci, _vp]),
    "fa_decode": (_ci, [_vp] * 6 + [_sz, _ci, _ci, _ci, _ci, _ci, _cf, _ci, _vp]),
    "fa_decode_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci]),
    "fa_decode_plan": (_ci, [_ci, _ci, _ci, _ci, _ci, _ci, ctypes.POINTER(_ci), ctypes.POINTER(_ci)]),
    "fa_kv_append": (_ci, [_vp, _vp, _ll, _ll, _vp, _vp, _ll, _ll, _ci, _vp, _vp, _ci, _vp, _vp, _ci, _ci,
                           _vp, _vp, _ci, _ci, _vp, _ci, _ci, _vp]),
    "fa_decode_paged": (_ci, [_vp, _vp, _vp, _vp, _ci, _vp, _vp, _vp, _vp, _vp, _sz, _ci, _ci, _ci,
                              _cf, _ci, _vp]),
    "fa_decode_paged_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci]),
    "fa_decode_shared": (_ci, [_vp, _vp, _vp, _vp, _ci, _vp, _ci, _vp, _vp, _vp, _vp, _vp, _sz, _ci,
                               _ci, _ci, _cf, _ci, _vp]),
    "fa_decode_shared_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci, _ci, _ci]),
    "fa_decode_shared_plan": (_ci, [_ci] * 9 + [ctypes.POINTER(_ci)] * 2),
    "fa_check_device_status": (_ci, [_vp]),
    "fa_debug_timeout_probe": (_ci, [ctypes.c_longlong, _vp]),
    "fa_debug_fwd_skip_load": (_ci, [_vp] * 5 + [_ci, _ci, _ci, _ci, _cf, _ci, ctypes.c_longlong, _vp]),
    "fa_debug_bwd_skip_load": (_ci, [_vp] * 10 + [_sz, _ci, _ci, _ci, _ci, _cf, _ci,
                                                  ctypes.c_longlong, _vp]),
    "fa_debug_bwd_skip_load_ex": (_ci, [_vp] * 10 + [_sz, _ci, _ci, _ci, _ci, _cf, _ci, _ci,
                                                     ctypes.c_longlong, _vp]),
    "fa_debug_decode_skip_load": (_ci, [_vp, _vp, _vp, _vp, _ci, _vp, _ci, _vp, _vp, _vp, _vp, _vp, _sz, _ci,
                                        _ci, _ci, _cf, _ci, _ll, _vp]),
    "fa_status_string": (ctypes.c_char_p, [_ci]),
    "fa_version": (_ci, []),
}


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {fa_status_string(code)}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load ``libfa_gb300.so`` (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with `python -m exact_attention_30_gb300.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def header_functions(header_path: str | None = None):
    """Names of the functions declared in include/fa.h (for export checks)."""
    path = header_path or os.path.join(os.path.dirname(_HERE), "include", "fa.h")
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", text)))


def fa_status_string(code: int) -> str:
    return load_library().fa_status_string(int(code)).decode()


def fa_version() -> int:
    return load_library().fa_version()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use torch.bfloat16 or torch.float32")


def _check(t: torch.Tensor, name: str, like: torch.Tensor | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [B,H,N,d]")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must match q in shape, dtype and device")


def _stream_ptr(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _raw_stream(index: int) -> int:
    """The current stream of device ``index``, without building a Stream object where torch allows."""
    return _get_raw_stream(index) if _get_raw_stream is not None else _stream_ptr(index)


def _raise(code: int, where: str):
    if code != FA_OK:
        raise FAError(code, where)


def fa_fwd_workspace_bytes(B: int, H: int, N: int, d: int, causal: bool = False,
                           dtype=torch.bfloat16) -> int:
    """Scratch bytes with which the forward splits its last, partly filled
    wave of CTAs on the current device (0: nothing to gain)."""
    code = FA_BF16 if dtype == torch.bfloat16 else FA_F32
    return int(load_library().fa_fwd_workspace_bytes(B, H, N, d, FA_CAUSAL if causal else 0, code))


def fa_fwd_plan(B: int, H: int, N: int, d: int, causal: bool = False, dtype=torch.bfloat16,
                resident_ctas: int = 0):
    """(n_full, n_tail, splits) of the forward's schedule (fa_fwd_plan in fa.h)."""
    nf, nt, sp = _ci(), _ci(), _ci()
    code = FA_BF16 if dtype == torch.bfloat16 else FA_F32
    rc = load_library().fa_fwd_plan(B, H, N, d, FA_CAUSAL if causal else 0, code, resident_ctas,
                                    ctypes.byref(nf), ctypes.byref(nt), ctypes.byref(sp))
    _raise(rc, "fa_fwd_plan")
    return nf.value, nt.value, sp.value


def fa_bwd_plan(B: int, H: int, N: int, d: int, causal: bool = False, dtype=torch.bfloat16,
                resident_ctas: int = 0):
    """(n_full, n_tail, splits) of the backward main kernel's schedule (fa_bwd_plan in fa.h)."""
    nf, nt, sp = _ci(), _ci(), _ci()
    code = FA_BF16 if dtype == torch.bfloat16 else FA_F32
    rc = load_library().fa_bwd_plan(B, H, N, d, FA_CAUSAL if causal else 0, code, resident_ctas,
                                    ctypes.byref(nf), ctypes.byref(nt), ctypes.byref(sp))
    _raise(rc, "fa_bwd_plan")
    return nf.value, nt.value, sp.value


def fa_fwd(q, k, v, scale: float | None = None, out=None, lse=None, causal: bool = False,
           workspace=None):
    """Forward pass: returns (O [B,H,N,d] like q, LSE [B,H,N] float32).

    When the problem gains from splitting the tail of the schedule
    (fa_fwd_workspace_bytes > 0), the scratch is allocated here unless a
    uint8 CUDA tensor of at least that size is passed as ``workspace``."""
    lib = load_library()
    _check(q, "q")
    _check(k, "k", q)
    _check(v, "v", q)
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "out", q)
    if lse.dtype != torch.float32 or lse.shape != (B, H, N) or not lse.is_cuda:
        raise ValueError("lse must be float32 [B,H,N] on the same device")
    flags = FA_CAUSAL if causal else 0
    with torch.cuda.device(q.device):
        ws_bytes = int(lib.fa_fwd_workspace_bytes(B, H, N, d, flags, _dtype_code(q)))
        if ws_bytes > 0 and workspace is None:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            if workspace.dtype != torch.uint8 or not workspace.is_cuda or workspace.device != q.device:
                raise ValueError("workspace must be a uint8 tensor on q's device")
            rc = lib.fa_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               workspace.data_ptr(), workspace.numel(), B, H, N, d, scale, flags,
                               _dtype_code(q), _stream_ptr(q.device))
        else:
            rc = lib.fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               B, H, N, d, scale, flags, _dtype_code(q), _stream_ptr(q.device))
    _raise(rc, "fa_fwd")
    return o, lse


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int, dtype=torch.bfloat16) -> int:
    code = FA_BF16 if dtype == torch.bfloat16 else FA_F32
    return int(load_library().fa_bwd_workspace_bytes(B, H, N, d, code))


def _bwd_call(stage, q, k, v, o, do, lse, scale, workspace, dq, dk, dv, causal=False):
    lib = load_library()
    _check(q, "q")
    for t, n in ((k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _check(t, n, q)
    B, H, N, d = q.shape
    if lse.dtype != torch.float32 or lse.shape != (B, H, N) or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B,H,N] on the same device")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if workspace is None:
        ws_bytes = fa_bwd_workspace_bytes(B, H, N, d, q.dtype)
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _check(t, n, q)
    if stage is not None and stage not in _STAGE_FLAGS:
        raise ValueError(f"unknown backward stage {stage}")
    flags = (FA_CAUSAL if causal else 0) | (0 if stage is None else _STAGE_FLAGS[stage])
    with torch.cuda.device(q.device):
        rc = lib.fa_bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                           lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           B, H, N, d, scale, flags, _dtype_code(q), _stream_ptr(q.device))
    _raise(rc, "fa_bwd" if stage is None else "fa_bwd_stage")
    return dq, dk, dv


def fa_bwd(q, k, v, o, do, lse, scale: float | None = None, workspace=None, dq=None, dk=None,
           dv=None, causal: bool = False):
    """Backward pass: returns (dQ, dK, dV), each like q."""
    return _bwd_call(None, q, k, v, o, do, lse, scale, workspace, dq, dk, dv, causal)


def fa_bwd_stage(stage: int, q, k, v, o, do, lse, scale: float | None = None, workspace=None,
                 dq=None, dk=None, dv=None, causal: bool = False):
    """One backward stage (FA_BWD_PREPROCESS, FA_BWD_MAIN, FA_BWD_DQ_CONVERT) on ``workspace``."""
    return _bwd_call(stage, q, k, v, o, do, lse, scale, workspace, dq, dk, dv, causal)


def _check_varlen(q, cu_seqlens, max_seqlen):
    _check(q, "q")
    if q.dim() != 3:
        raise ValueError("packed tensors are [total, H, d]")
    if not isinstance(cu_seqlens, torch.Tensor) or not cu_seqlens.is_cuda or \
            cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor [B+1]")
    if cu_seqlens.device != q.device:
        raise ValueError("cu_seqlens must be on q's device")
    total, H, d = q.shape
    return cu_seqlens.numel() - 1, H, total, int(max_seqlen), d


def fa_bwd_varlen_workspace_bytes(B: int, H: int, total: int, max_seqlen: int, d: int,
                                  dtype=torch.bfloat16) -> int:
    code = FA_BF16 if dtype == torch.bfloat16 else FA_F32
    return int(load_library().fa_bwd_varlen_workspace_bytes(B, H, total, max_seqlen, d, code))


def fa_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, scale: float | None = None,
                  causal: bool = False, out=None, lse=None):
    """Packed variable-length forward: q, k, v [total, H, d]; cu_seqlens int32 [B+1] on the GPU.

    Returns (O [total, H, d] like q, LSE [H, total] float32).
    """
    lib = load_library()
    B, H, total, max_seqlen, d = _check_varlen(q, cu_seqlens, max_seqlen)
    _check(k, "k", q)
    _check(v, "v", q)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((H, total), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "out", q)
    if lse.dtype != torch.float32 or lse.shape != (H, total) or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [H, total] on the same device")
    with torch.cuda.device(q.device):
        rc = lib.fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               cu_seqlens.data_ptr(), B, H, total, max_seqlen, d, scale,
                               FA_CAUSAL if causal else 0, _dtype_code(q), _stream_ptr(q.device))
    _raise(rc, "fa_fwd_varlen")
    return o, lse


def fa_bwd_varlen(q, k, v, o, do, lse, cu_seqlens, max_seqlen: int, scale: float | None = None,
                  causal: bool = False, workspace=None):
    """Backward of ``fa_fwd_varlen``: returns (dQ, dK, dV), each [total, H, d] like q."""
    lib = load_library()
    B, H, total, max_seqlen, d = _check_varlen(q, cu_seqlens, max_seqlen)
    for t, n in ((k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _check(t, n, q)
    if lse.dtype != torch.float32 or lse.shape != (H, total) or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [H, total] on the same device")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    with torch.cuda.device(q.device):
        if workspace is None:
            n = fa_bwd_varlen_workspace_bytes(B, H, total, max_seqlen, d, q.dtype)
            workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
        rc = lib.fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                               lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                               cu_seqlens.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), B, H, total, max_seqlen,
                               d, scale, FA_CAUSAL if causal else 0, _dtype_code(q),
                               _stream_ptr(q.device))
    _raise(rc, "fa_bwd_varlen")
    return dq, dk, dv


def fa_softmax_rows(x, scale: float = 1.0, out=None):
    """Row softmax of a CUDA tensor (last dimension = row), fp32 or bf16; returns ``out``."""
    lib = load_library()
    _check(x, "x")
    cols = x.shape[-1]
    rows = x.numel() // max(cols, 1)
    y = torch.empty_like(x) if out is None else out
    _check(y, "out", x)
    with torch.cuda.device(x.device):
        rc = lib.fa_softmax_rows(x.data_ptr(), y.data_ptr(), rows, cols, float(scale),
                                 _dtype_code(x), _stream_ptr(x.device))
    _raise(rc, "fa_softmax_rows")
    return y


def fa_decode_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int, dtype=torch.bfloat16) -> int:
    """Scratch bytes fa_decode needs on the current device."""
    code = FA_BF16 if dtype == torch.bfloat16 else FA_F32
    return int(load_library().fa_decode_workspace_bytes(B, H, Nq, Nk, d, code))


def fa_decode_plan(B: int, H: int, Nq: int, Nk: int, d: int, resident_ctas: int = 0):
    """(splits, keys_per_split) that fa_decode uses; resident_ctas > 0 plans without a device."""
    s, k = ctypes.c_int(0), ctypes.c_int(0)
    _raise(load_library().fa_decode_plan(B, H, Nq, Nk, d, int(resident_ctas), ctypes.byref(s),
                                         ctypes.byref(k)), "fa_decode_plan")
    return s.value, k.value


def fa_decode(q, k, v, scale: float | None = None, out=None, lse=None, workspace=None):
    """KV-cache decode: q [B,H,Nq,d] (Nq <= 16) against k, v [B,H,Nk,d], bf16.

    Returns (O like q, LSE [B,H,Nq] float32).
    """
    lib = load_library()
    _check(q, "q")
    _check(k, "k")
    _check(v, "v", k)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,Nq,d] and k, v [B,H,Nk,d]")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape[0] != B or k.shape[1] != H or k.shape[3] != d or k.dtype != q.dtype or k.device != q.device:
        raise ValueError("k, v must be [B,H,Nk,d] with q's B, H, d, dtype and device")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(o, "out", q)
    if lse.dtype != torch.float32 or lse.shape != (B, H, Nq) or not lse.is_cuda or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B,H,Nq] on the same device")
    with torch.cuda.device(q.device):
        if workspace is None:
            ws_bytes = fa_decode_workspace_bytes(B, H, Nq, Nk, d, q.dtype)
            workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
        rc = lib.fa_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                           B, H, Nq, Nk, d, scale, _dtype_code(q), _stream_ptr(q.device))
    _raise(rc, "fa_decode")
    return o, lse


def fa_rope_tables(max_positions: int, rot_dim: int, base: float = 10000.0, device=None):
    """Cosines and sines (float32 [max_positions, rot_dim / 2]) of the angles
    p * base^(-2i / rot_dim), computed in float64 (far positions) and rounded once."""
    if rot_dim < 2 or rot_dim % 2 != 0 or max_positions < 1:
        raise ValueError("rot_dim must be even and positive, max_positions positive")
    f = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * f
    return a.cos().float(), a.sin().float()


_BF16, _F32, _I32, _Tensor = torch.bfloat16, torch.float32, torch.int32, torch.Tensor


def _refuse(t, name: str, device: int, dtype, what: str):
    """Raises for argument ``name``, which is not what the caller's test asks for."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    raise ValueError(f"{name} must be {what}, {dtype}, on the other tensors' device (cuda:{device}); "
                     f"it is {tuple(t.shape)}, {t.dtype}, on {t.device}")


def _int32(n: int, name: str) -> int:
    """n, which the library takes as a C int; ctypes would cut it to 32 bits without a word."""
    if not -(1 << 31) <= n < 1 << 31:
        raise ValueError(f"{name} = {n} does not fit 32 bits")
    return n


def _is(t, dtype, device: int) -> bool:
    """Whether t is a tensor of ``dtype`` on CUDA device ``device``."""
    return isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device


def _paged_cache(k_pages, v_pages, block_tables, seq_lens):
    """Checks a paged cache and its tables; returns (fa_paged_kv, its shape, B, max_pages, device index)."""
    dev = k_pages.get_device() if isinstance(k_pages, _Tensor) else -1
    if dev < 0 or not _is(k_pages, _BF16, dev) or k_pages.dim() != 4:
        _refuse(k_pages, "k_pages", dev, _BF16, "[pages, Hkv, page_size, d]")
    shape = k_pages.shape
    if not _is(v_pages, _BF16, dev) or v_pages.shape != shape:
        _refuse(v_pages, "v_pages", dev, _BF16, "of k_pages' shape")
    if not _is(block_tables, _I32, dev) or block_tables.dim() != 2 or not block_tables.is_contiguous():
        _refuse(block_tables, "block_tables", dev, _I32, "a contiguous [B, max_pages]")
    B, max_pages = block_tables.shape
    _int32(max_pages, "the width of block_tables")
    if not _is(seq_lens, _I32, dev) or seq_lens.shape != (B,) or not seq_lens.is_contiguous():
        _refuse(seq_lens, "seq_lens", dev, _I32, "a contiguous [B]")
    k0, k1, k2, k3 = k_pages.stride()
    v0, v1, v2, v3 = v_pages.stride()
    if k3 != 1 or v3 != 1:
        raise ValueError("the last dimension of k_pages and v_pages must be contiguous")
    pool = _pack_pool(k_pages.data_ptr(), v_pages.data_ptr(), *shape, k0, k1, k2, v0, v1, v2)
    return pool, shape, B, max_pages, dev


def _on_device(dev: int, fn, *args):
    """fn(*args, current stream of device dev), with dev as the current device."""
    if dev == _current_device():  # a CUDA tensor is there, so CUDA is initialised
        return fn(*args, _raw_stream(dev))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(dev))


def _token_stride(t, name: str, total, heads, d: int, dev: int):
    """Checks packed tokens [total, heads, d] (heads of a token contiguous); returns their stride."""
    if not _is(t, _BF16, dev) or t.dim() != 3:
        _refuse(t, name, dev, _BF16, f"[total, heads, {d}]")
    n, h, e = t.shape
    s0, s1, s2 = t.stride()
    if e != d or (heads is not None and h != heads) or (total is not None and n != total):
        raise ValueError(f"{name} must be [total, heads, {d}] with the other tensors' tokens and heads")
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return s0


def fa_kv_append(k, v, k_pages, v_pages, block_tables, seq_lens, cu_seqlens=None, q=None, cos=None, sin=None,
                 interleaved: bool = False, positions=None, q_out=None):
    """Append new keys and values to a paged cache, rotating the keys (and q) by their position.

    k, v: [total, Hkv, d] bf16 packed new tokens (a slice of a fused projection
    will do); q: [total, Hq, d] or None. cu_seqlens: int32 [B+1] offsets of the
    sequences' new tokens (None: total / B tokens each); tokens outside all of
    them are padding. seq_lens: int32 [B] lengths after this append. cos, sin: float32 [max_positions, rot_dim / 2]
    (None: no rotation). positions: int32 [total] rotary positions (None: the
    key's index in the cache). k_pages and v_pages are written in place.
    Returns the rotated queries (``q_out``, dense unless given), or None without q.
    """
    pool, (_, hkv, page, d), B, max_pages, dev = _paged_cache(k_pages, v_pages, block_tables, seq_lens)
    ks = _token_stride(k, "k", None, hkv, d, dev)
    total = k.shape[0]
    vs = _token_stride(v, "v", total, hkv, d, dev)
    hq = qs = os_ = 0
    q_ptr = out_ptr = cu_ptr = cos_ptr = sin_ptr = pos_ptr = None
    if q is not None:
        qs = _token_stride(q, "q", total, None, d, dev)
        hq = q.shape[1]
        if q_out is None:
            q_out = torch.empty((total, hq, d), dtype=_BF16, device=q.device)
            os_ = hq * d
        else:
            os_ = _token_stride(q_out, "q_out", total, hq, d, dev)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out given without q")
    if cu_seqlens is not None:
        if not _is(cu_seqlens, _I32, dev) or cu_seqlens.shape != (B + 1,) or not cu_seqlens.is_contiguous():
            _refuse(cu_seqlens, "cu_seqlens", dev, _I32, "a contiguous [B+1]")
        cu_ptr = cu_seqlens.data_ptr()
    rot = max_pos = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if not _is(cos, _F32, dev) or cos.dim() != 2 or not cos.is_contiguous():
            _refuse(cos, "cos", dev, _F32, "a contiguous [max_positions, rot_dim / 2]")
        max_pos, rot = cos.shape
        if not _is(sin, _F32, dev) or sin.shape != (max_pos, rot) or not sin.is_contiguous():
            _refuse(sin, "sin", dev, _F32, "contiguous and of cos' shape")
        rot *= 2
        cos_ptr, sin_ptr = cos.data_ptr(), sin.data_ptr()
    if positions is not None:
        if not _is(positions, _I32, dev) or positions.shape != (total,) or not positions.is_contiguous():
            _refuse(positions, "positions", dev, _I32, "a contiguous [total]")
        pos_ptr = positions.data_ptr()
    if total == 0:
        return q_out
    rc = _on_device(dev, load_library().fa_kv_append, k.data_ptr(), v.data_ptr(), ks, vs, q_ptr, out_ptr, qs, os_, hq,
                    pool, block_tables.data_ptr(), max_pages, seq_lens.data_ptr(), cu_ptr, B, total, cos_ptr, sin_ptr,
                    rot, max_pos, pos_ptr, FA_ROPE_INTERLEAVED if interleaved else 0, FA_BF16)
    if rc != FA_OK:
        _raise(rc, "fa_kv_append")
    return q_out


def fa_decode_paged_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    """Scratch bytes fa_decode_paged needs on the current device."""
    return int(load_library().fa_decode_paged_workspace_bytes(B, Hq, Hkv, Nq, d, FA_BF16))


def fa_decode_shared_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, prefix_len: int, d: int) -> int:
    """Scratch bytes fa_decode_shared needs on the current device."""
    prefix_len = _int32(int(prefix_len), "prefix_len")
    return int(load_library().fa_decode_shared_workspace_bytes(B, Hq, Hkv, Nq, prefix_len, d, FA_BF16))


def fa_decode_shared_plan(B: int, Hq: int, Hkv: int, Nq: int, prefix_len: int, d: int, page_size: int, max_pages: int,
                          sms: int = 0):
    """(key ranges, CTAs) of the prefix's kernel in fa_decode_shared, (0, 0) if it has none; sms > 0 plans without a device."""
    ranges, ctas = ctypes.c_int(0), ctypes.c_int(0)
    prefix_len, max_pages = _int32(int(prefix_len), "prefix_len"), _int32(max_pages, "max_pages")
    _raise(load_library().fa_decode_shared_plan(B, Hq, Hkv, Nq, prefix_len, d, page_size, max_pages, int(sms),
                                                ctypes.byref(ranges), ctypes.byref(ctas)), "fa_decode_shared_plan")
    return ranges.value, ctas.value


_decode_ws_bytes: dict = {}  # (device, sizes) -> bytes: what the library answered
_decode_scratch = threading.local()  # .by_device: device -> scratch of this thread's calls on the default stream
_SCRATCH_KEPT_BYTES = 64 << 20


def _decode_workspace(lib, key, device, stream: int):
    """Scratch for one call. Calls on the default stream (which is never
    captured and runs one after another) reuse one tensor per thread and device:
    allocating and freeing it took 5 of a call's 23 us. It is given back when the
    thread ends. Other streams, and calls that need more than 64 MB, get their own."""
    n = _decode_ws_bytes.get(key)
    if n is None:
        n = _decode_workspace_size(lib, key)
    if stream != 0 or n > _SCRATCH_KEPT_BYTES:
        return torch.empty(n, dtype=torch.uint8, device=device), n
    kept = _decode_scratch.__dict__.setdefault("by_device", {})
    w = kept.get(key[0])
    if w is None or w.shape[0] < n:
        kept[key[0]] = w = torch.empty(n, dtype=torch.uint8, device=device)
    return w, w.shape[0]


def _decode_workspace_size(lib, key):
    dev, B, hq, hkv, nq, prefix_len, d = key
    with torch.cuda.device(dev):
        n = lib.fa_decode_shared_workspace_bytes(B, hq, hkv, nq, prefix_len, d, FA_BF16)
    if len(_decode_ws_bytes) >= 4096:
        _decode_ws_bytes.clear()
    _decode_ws_bytes[key] = n
    return n


def _decode_cache(where, q, k_pages, v_pages, prefix_pages, prefix_len, block_tables, seq_lens, scale, out, lse,
                  workspace):
    lib = load_library()
    pool, (_, hkv, page, d), B, max_pages, dev = _paged_cache(k_pages, v_pages, block_tables, seq_lens)
    if not _is(q, _BF16, dev) or q.dim() != 4:
        _refuse(q, "q", dev, _BF16, "[B, Hq, Nq, d]")
    shape = q.shape
    b, hq, nq, e = shape
    if b != B or e != d or hq % hkv != 0:
        raise ValueError("q must be [B, Hq, Nq, d] with the tables' B, the cache's d and Hq a multiple of its heads")
    q0, q1, q2, q3 = q.stride()
    device = q.device
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=device)
        o_strides, o3 = None, 1
    else:
        if not _is(out, _BF16, dev) or out.shape != shape:
            _refuse(out, "out", dev, _BF16, "of q's shape")
        o0, o1, o2, o3 = out.stride()
        o_strides = _pack_strides(o0, o1, o2)
    if q3 != 1 or o3 != 1:
        raise ValueError("the last dimension of q and out must be contiguous")
    if lse is None:
        lse = torch.empty((B, hq, nq), dtype=_F32, device=device)
    elif not _is(lse, _F32, dev) or lse.shape != (B, hq, nq) or not lse.is_contiguous():
        _refuse(lse, "lse", dev, _F32, "a contiguous [B, Hq, Nq]")
    prefix_ptr = None
    if prefix_len > 0:
        if not _is(prefix_pages, _I32, dev) or prefix_pages.dim() != 1 or not prefix_pages.is_contiguous():
            _refuse(prefix_pages, "prefix_pages", dev, _I32, "a contiguous [pages]")
        if prefix_pages.shape[0] * page < prefix_len:
            raise ValueError("prefix_pages holds fewer than prefix_len keys")
        prefix_ptr = prefix_pages.data_ptr()
    if workspace is None:
        workspace, n = _decode_workspace(lib, (dev, B, hq, hkv, nq, prefix_len, d), device, _raw_stream(dev))
    else:
        if not isinstance(workspace, _Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        n = workspace.numel() * workspace.element_size()
    rc = _on_device(dev, lib.fa_decode_shared, q.data_ptr(), _pack_strides(q0, q1, q2), pool, prefix_ptr, prefix_len,
                    block_tables.data_ptr(), max_pages, seq_lens.data_ptr(), out.data_ptr(), o_strides,
                    lse.data_ptr(), workspace.data_ptr(), n, B, hq, nq, scale, FA_BF16)
    if rc != FA_OK:
        _raise(rc, where)
    return out, lse


def fa_decode_paged(q, k_pages, v_pages, block_tables, seq_lens, scale: float | None = None, out=None, lse=None,
                    workspace=None):
    """Decode against a paged cache: the Nq newest tokens of each sequence over its seq_lens[b] keys.

    q: [B, Hq, Nq, d] bf16, any strides with d contiguous (Hq / Hkv * Nq <= 64);
    k_pages, v_pages: [pages, Hkv, page_size, d] bf16, any strides with d
    contiguous; block_tables int32 [B, max_pages]; seq_lens int32 [B]. Query i
    sees keys j < seq_lens[b] - Nq + 1 + i; one that sees none gets O = 0 and
    LSE = -inf. Returns (O like q, LSE [B, Hq, Nq] float32).
    """
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    return _decode_cache("fa_decode_paged", q, k_pages, v_pages, None, 0, block_tables, seq_lens, scale, out, lse,
                         workspace)


def fa_decode_shared(q, k_pages, v_pages, prefix_pages, prefix_len: int, block_tables, seq_lens,
                     scale: float | None = None, out=None, lse=None, workspace=None):
    """``fa_decode_paged`` for a batch whose sequences all continue one prefix.

    prefix_pages: int32 [ceil(prefix_len / page_size)] pages of the prefix, loaded
    once per 256 query rows of a K/V head; block_tables and seq_lens describe the sequences'
    own keys, which follow the prefix. Returns (O like q, LSE [B, Hq, Nq] float32).
    """
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else float(scale)
    prefix_len = _int32(int(prefix_len), "prefix_len")
    if prefix_len > 0 and prefix_pages is None:
        raise ValueError("prefix_pages is missing")
    return _decode_cache("fa_decode_shared", q, k_pages, v_pages, prefix_pages, prefix_len, block_tables, seq_lens,
                         scale, out, lse, workspace)


def fa_check_device_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device status code."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(load_library().fa_check_device_status(_stream_ptr(dev)))


def fa_debug_timeout_probe(limit_ns: int, device=None) -> int:
    """Launch the bounded-wait probe kernel (see include/fa.h); returns the launch status."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(load_library().fa_debug_timeout_probe(int(limit_ns), _stream_ptr(dev)))
