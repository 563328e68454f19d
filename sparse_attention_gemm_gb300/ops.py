"""Thin Python binding of libdsa.so (include/dsa.h), same entry-point names.

Argument marshalling only: tensors are checked for device, dtype and
contiguity, outputs are allocated with torch (device memory is the caller's
business on the C side), and every call goes straight to the C ABI on the
current torch stream.  Every step of the path runs in the library's CUDA
kernels; there is no fallback.  If the library is missing, the first call
raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# DSA_LIB_PATH selects another build of this library (the range-checked one
# under _build_checked/, for its tests); by default the optimised build.
LIB_PATH = os.environ.get("DSA_LIB_PATH") or os.path.join(_HERE, "_build", "libdsa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "dsa.h")

DSA_OK = 0
DSA_ERR_VALUE = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_CUDA = 3
DSA_ERR_WORKSPACE = 4
DSA_STATUS_WAIT_TIMEOUT = 0x1
DSA_STATUS_CAND_OVERFLOW = 0x2
DSA_STATUS_DRAIN_TIMEOUT = 0x4
DSA_STATUS_CHECK_FAILED = 0x8
MAX_TOPK = 2048

_lock = threading.Lock()
_lib = None

P = ctypes.c_void_p
I = ctypes.c_int
I64 = ctypes.c_int64
F = ctypes.c_float
D = ctypes.c_double
SZ = ctypes.c_size_t

_SIGNATURES = {
    "dsa_last_error": ([], ctypes.c_char_p),
    "dsa_device_status": ([P, I], I),
    "dsa_set_wait_limit_ns": ([ctypes.c_uint64], I),
    "dsa_thd_metadata": ([P, I, I, P, P, P], I),
    "dsa_indexer_scores": ([P, P, P, P, I, I, I, I, I, P, I64, P], I),
    "dsa_topk": ([P, I64, P, P, I, I, P, P, P, P], I),
    "dsa_compact_sort_indices": ([P, I, I, I64, P, P, P], I),
    "dsa_indexer_topk_workspace_size": ([I, I, I, I, I], SZ),
    "dsa_indexer_topk": ([P, P, P, P, I, I, I, I, I, I, P, P, P, SZ, P], I),
    "dsa_indexer_topk_ex": ([P, P, P, P, I, I, I, I, I, I, P, P, P, P, P, P, SZ, P], I),
    "dsa_topk_softmax": ([P, P, I, I, P, P, P], I),
    "dsa_forward_host": ([P, I, I, I, I, I, I, I, I, I, F, I, P, P], I),
    "dsa_indexer_topk_noalloc": ([P, P, P, P, I, I, I, I, I, I, P, P, P], I),
    "dsa_indexer_candidates": ([P, P, P, P, I, I, I, I, I, I, P, SZ, P], I),
    "dsa_select_candidates": ([P, I, I, I, I, I, I, P, SZ, P, P, P], I),
    "dsa_sparse_attn_fwd": ([P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, P], I),
    "dsa_sparse_attn_fwd_ex": ([P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, I, P, P], I),
    "dsa_pack_routes": ([P, I, I, I, P, P], I),
    "dsa_thd_metadata_ratio": ([P, P, P, I, I, I, P, P, P], I),
    "dsa_indexer_scores_ratio": ([P, P, P, P, P, P, I, I, I, I, I, I, I, P, I64, P], I),
    "dsa_indexer_topk_ratio": ([P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P, P, SZ, P], I),
    "dsa_indexer_scores_fp8": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, I64, P], I),
    "dsa_indexer_topk_fp8": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P, P, SZ, P], I),
    "dsa_indexer_scores_mxfp8": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, I64, P], I),
    "dsa_indexer_topk_mxfp8": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P, P, SZ, P], I),
    "dsa_sparse_attn_bwd_workspace_size": ([I, I, I, I], SZ),
    "dsa_sparse_attn_bwd": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, SZ, P], I),
    "dsa_sparse_attn_bwd_workspace_size_ex": ([I, I, I, I, I], SZ),
    "dsa_kv8_write": ([P, P, P, P, I, I, I, I, I, I, I, P, P, P], I),
    "dsa_kv8_read": ([P, P, P, P, P, I, I, I, I, I, I, I, P, P], I),
    "dsa_sparse_attn_fwd_kv8_workspace_size": ([I, I, I, I, I, I], SZ),
    "dsa_sparse_attn_fwd_kv8": ([P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, P, P, P, P, P, SZ, P], I),
    "dsa_kv4_write": ([P, P, P, P, I, I, I, I, I, I, I, P, P, P], I),
    "dsa_kv4_read": ([P, P, P, P, P, I, I, I, I, I, I, I, P, P], I),
    "dsa_sparse_attn_fwd_kv4_workspace_size": ([I, I, I, I, I, I, I, I, I], SZ),
    "dsa_sparse_attn_fwd_kv4": ([P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, P, P, P, P, P, SZ, P], I),
    "dsa_rms_norm_fwd": ([P, I64, P, I64, P, I, I, F, I, P, I64, P, P, I64, P, P], I),
    "dsa_rms_norm_bwd_workspace_size": ([I, I], SZ),
    "dsa_rms_norm_bwd": ([P, I64, P, I64, P, P, P, I64, I, I, P, I64, P, P, SZ, P], I),
    "dsa_rotary": ([P, I64, I64, I, P, I64, I64, I, P, P, P, I, I, I, I, I, F, P, I64, I64, P, I64, I64, P], I),
    "dsa_rotary_inv_freq": ([I, D, I, D, I64, D, D, P, P], I),
    "dsa_sparse_attn_bwd_ex": ([P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, I, P, SZ, P], I),
}


class DsaError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed ({code}): {msg}")
        self.code = code


def header_functions() -> list[str]:
    """Names of the functions that include/dsa.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w\s\*]*?\b(dsa_\w+)\s*\(", text, re.M)))


def lib() -> ctypes.CDLL:
    """The loaded libdsa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libdsa.so is not built ({LIB_PATH}); run __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGNATURES.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _lib = L
    return _lib


def _check(fn: str, rc: int) -> None:
    if rc != DSA_OK:
        msg = lib().dsa_last_error().decode(errors="replace")
        if rc in (DSA_ERR_VALUE, DSA_ERR_WORKSPACE):
            raise ValueError(f"{fn}: {msg}")
        raise DsaError(fn, rc, msg)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, name, dtype, dim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    return t


def device_status(clear: bool = True) -> int:
    v = ctypes.c_uint32(0)
    _check("dsa_device_status", lib().dsa_device_status(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


def set_wait_limit_ns(limit_ns: int) -> None:
    """Bounded-wait limit of the kernels launched afterwards on the current
    device (0: the library default).  Failure-detection hook; synchronises."""
    _check("dsa_set_wait_limit_ns", lib().dsa_set_wait_limit_ns(int(limit_ns)))


def thd_metadata(cu_seqlens: torch.Tensor, T: int):
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    start = torch.empty(T, dtype=torch.int32, device=cu_seqlens.device)
    length = torch.empty(T, dtype=torch.int32, device=cu_seqlens.device)
    _check("dsa_thd_metadata", lib().dsa_thd_metadata(_p(cu_seqlens), cu_seqlens.numel() - 1, T, _p(start),
                                                      _p(length), _stream()))
    return start, length


def thd_metadata_ratio(cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int, T: int):
    """start, len [T] of the ratio-causal compressed-key mask."""
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    if q_causal_offsets is not None:
        _need(q_causal_offsets, "q_causal_offsets", torch.int32, 1)
    start = torch.empty(T, dtype=torch.int32, device=cu_seqlens_q.device)
    length = torch.empty(T, dtype=torch.int32, device=cu_seqlens_q.device)
    _check("dsa_thd_metadata_ratio",
           lib().dsa_thd_metadata_ratio(_p(cu_seqlens_q), _p(cu_seqlens_k), _p(q_causal_offsets),
                                        cu_seqlens_q.numel() - 1, T, int(ratio), _p(start), _p(length), _stream()))
    return start, length


def _ratio_inputs(qi, ki, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets):
    _need(qi, "qi", torch.bfloat16, 3)
    _need(ki, "ki", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    if q_causal_offsets is not None:
        _need(q_causal_offsets, "q_causal_offsets", torch.int32, 1)
    if cu_seqlens_k.numel() != cu_seqlens_q.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    return qi.shape[0], ki.shape[0], qi.shape[1], qi.shape[2]


def indexer_scores_ratio(qi, ki, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int, s_max: int,
                         ld: int | None = None, out=None):
    """Dense compressed-key indexer scores fp32 [Tq, ld] under the ratio-causal mask."""
    Tq, Tk, Hi, d = _ratio_inputs(qi, ki, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets)
    ld = ld or (s_max + 3) // 4 * 4
    if out is None:
        out = torch.empty((Tq, ld), dtype=torch.float32, device=qi.device)
    _check("dsa_indexer_scores_ratio",
           lib().dsa_indexer_scores_ratio(_p(qi), _p(ki), _p(w), _p(cu_seqlens_q), _p(cu_seqlens_k),
                                          _p(q_causal_offsets), cu_seqlens_q.numel() - 1, Tq, Tk, Hi, d, int(ratio),
                                          s_max, _p(out), ld, _stream()))
    return out


def indexer_topk_ratio(qi, ki, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int, k: int, s_max: int,
                       want_logits: bool = False, want_softmax: bool = False, want_lse: bool = False, workspace=None):
    """Combined compressed-key indexer + top-k: dict(idx [Tq, k] ascending
    global key rows, topk_length[, logits][, softmax][, lse])."""
    Tq, Tk, Hi, d = _ratio_inputs(qi, ki, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets)
    dev = qi.device
    if workspace is None:
        workspace = torch.empty(indexer_topk_workspace_size(Tq, Hi, d, k, s_max), dtype=torch.uint8, device=dev)
    want_logits = want_logits or want_softmax or want_lse
    idx = torch.empty((Tq, k), dtype=torch.int32, device=dev)
    tl = torch.empty(Tq, dtype=torch.int32, device=dev)
    logits = torch.empty((Tq, k), dtype=torch.float32, device=dev) if want_logits else None
    sm = torch.empty((Tq, k), dtype=torch.float32, device=dev) if want_softmax else None
    lse = torch.empty(Tq, dtype=torch.float32, device=dev) if want_lse else None
    _check("dsa_indexer_topk_ratio",
           lib().dsa_indexer_topk_ratio(_p(qi), _p(ki), _p(w), _p(cu_seqlens_q), _p(cu_seqlens_k),
                                        _p(q_causal_offsets), cu_seqlens_q.numel() - 1, Tq, Tk, Hi, d, int(ratio), k,
                                        s_max, _p(idx), _p(tl), _p(logits), _p(sm), _p(lse), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _stream()))
    res = {"idx": idx, "topk_length": tl}
    for name, t in (("logits", logits), ("softmax", sm), ("lse", lse)):
        if t is not None:
            res[name] = t
    return res


def _fp8_inputs(qi8, ki8, q_scale, k_scale, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets):
    _need(qi8, "qi8", torch.uint8, 3)
    _need(ki8, "ki8", torch.uint8, 2)
    _need(q_scale, "q_scale", torch.float32, 2)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    if q_causal_offsets is not None:
        _need(q_causal_offsets, "q_causal_offsets", torch.int32, 1)
    return qi8.shape[0], ki8.shape[0], qi8.shape[1], qi8.shape[2]


def indexer_scores_fp8(qi8, ki8, q_scale, k_scale, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int,
                       s_max: int, ld: int | None = None, out=None):
    """Dense indexer scores fp32 [Tq, ld] from E4M3 qi8 / ki8 (uint8 codes) and fp32 descales."""
    Tq, Tk, Hi, d = _fp8_inputs(qi8, ki8, q_scale, k_scale, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets)
    ld = ld or (s_max + 3) // 4 * 4
    if out is None:
        out = torch.empty((Tq, ld), dtype=torch.float32, device=qi8.device)
    _check("dsa_indexer_scores_fp8",
           lib().dsa_indexer_scores_fp8(_p(qi8), _p(ki8), _p(q_scale), _p(k_scale), _p(w), _p(cu_seqlens_q),
                                        _p(cu_seqlens_k), _p(q_causal_offsets), cu_seqlens_q.numel() - 1, Tq, Tk, Hi,
                                        d, int(ratio), s_max, _p(out), ld, _stream()))
    return out


def indexer_topk_fp8(qi8, ki8, q_scale, k_scale, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int, k: int,
                     s_max: int, want_logits: bool = False, want_softmax: bool = False, want_lse: bool = False,
                     workspace=None, idx=None, topk_length=None):
    """Combined indexer + top-k on E4M3 inputs: dict(idx, topk_length[, logits][, softmax][, lse])."""
    Tq, Tk, Hi, d = _fp8_inputs(qi8, ki8, q_scale, k_scale, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets)
    dev = qi8.device
    if workspace is None:
        workspace = torch.empty(indexer_topk_workspace_size(Tq, Hi, d, k, s_max), dtype=torch.uint8, device=dev)
    want_logits = want_logits or want_softmax or want_lse
    idx = torch.empty((Tq, k), dtype=torch.int32, device=dev) if idx is None else idx
    tl = torch.empty(Tq, dtype=torch.int32, device=dev) if topk_length is None else topk_length
    logits = torch.empty((Tq, k), dtype=torch.float32, device=dev) if want_logits else None
    sm = torch.empty((Tq, k), dtype=torch.float32, device=dev) if want_softmax else None
    lse = torch.empty(Tq, dtype=torch.float32, device=dev) if want_lse else None
    _check("dsa_indexer_topk_fp8",
           lib().dsa_indexer_topk_fp8(_p(qi8), _p(ki8), _p(q_scale), _p(k_scale), _p(w), _p(cu_seqlens_q),
                                      _p(cu_seqlens_k), _p(q_causal_offsets), cu_seqlens_q.numel() - 1, Tq, Tk, Hi, d,
                                      int(ratio), k, s_max, _p(idx), _p(tl), _p(logits), _p(sm), _p(lse),
                                      _p(workspace), workspace.numel() * workspace.element_size(), _stream()))
    res = {"idx": idx, "topk_length": tl}
    for name, t in (("logits", logits), ("softmax", sm), ("lse", lse)):
        if t is not None:
            res[name] = t
    return res


def _mxfp8_inputs(qi8, ki8, q_sf, k_sf, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets):
    _need(qi8, "qi8", torch.uint8, 3)
    _need(ki8, "ki8", torch.uint8, 2)
    _need(q_sf, "q_sf", torch.uint8, 3)
    _need(k_sf, "k_sf", torch.uint8, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    if q_causal_offsets is not None:
        _need(q_causal_offsets, "q_causal_offsets", torch.int32, 1)
    if q_sf.shape != (qi8.shape[0], qi8.shape[1], qi8.shape[2] // 32) or k_sf.shape != (ki8.shape[0], ki8.shape[1] // 32):
        raise ValueError("q_sf / k_sf must hold one scale byte per 32 elements of qi8 / ki8")
    return qi8.shape[0], ki8.shape[0], qi8.shape[1], qi8.shape[2]


def indexer_scores_mxfp8(qi8, ki8, q_sf, k_sf, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int,
                         s_max: int, ld: int | None = None, out=None):
    """Dense indexer scores fp32 [Tq, ld] from E4M3 qi8 / ki8 with E8M0 block scales q_sf / k_sf (uint8)."""
    Tq, Tk, Hi, d = _mxfp8_inputs(qi8, ki8, q_sf, k_sf, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets)
    ld = ld or (s_max + 3) // 4 * 4
    if out is None:
        out = torch.empty((Tq, ld), dtype=torch.float32, device=qi8.device)
    _check("dsa_indexer_scores_mxfp8",
           lib().dsa_indexer_scores_mxfp8(_p(qi8), _p(ki8), _p(q_sf), _p(k_sf), _p(w), _p(cu_seqlens_q),
                                          _p(cu_seqlens_k), _p(q_causal_offsets), cu_seqlens_q.numel() - 1, Tq, Tk,
                                          Hi, d, int(ratio), s_max, _p(out), ld, _stream()))
    return out


def indexer_topk_mxfp8(qi8, ki8, q_sf, k_sf, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets, ratio: int, k: int,
                       s_max: int, want_logits: bool = False, want_softmax: bool = False, want_lse: bool = False,
                       workspace=None, idx=None, topk_length=None):
    """Combined indexer + top-k on MXFP8 inputs: dict(idx, topk_length[, logits][, softmax][, lse])."""
    Tq, Tk, Hi, d = _mxfp8_inputs(qi8, ki8, q_sf, k_sf, w, cu_seqlens_q, cu_seqlens_k, q_causal_offsets)
    dev = qi8.device
    if workspace is None:
        workspace = torch.empty(indexer_topk_workspace_size(Tq, Hi, d, k, s_max), dtype=torch.uint8, device=dev)
    want_logits = want_logits or want_softmax or want_lse
    idx = torch.empty((Tq, k), dtype=torch.int32, device=dev) if idx is None else idx
    tl = torch.empty(Tq, dtype=torch.int32, device=dev) if topk_length is None else topk_length
    logits = torch.empty((Tq, k), dtype=torch.float32, device=dev) if want_logits else None
    sm = torch.empty((Tq, k), dtype=torch.float32, device=dev) if want_softmax else None
    lse = torch.empty(Tq, dtype=torch.float32, device=dev) if want_lse else None
    _check("dsa_indexer_topk_mxfp8",
           lib().dsa_indexer_topk_mxfp8(_p(qi8), _p(ki8), _p(q_sf), _p(k_sf), _p(w), _p(cu_seqlens_q),
                                        _p(cu_seqlens_k), _p(q_causal_offsets), cu_seqlens_q.numel() - 1, Tq, Tk, Hi,
                                        d, int(ratio), k, s_max, _p(idx), _p(tl), _p(logits), _p(sm), _p(lse),
                                        _p(workspace), workspace.numel() * workspace.element_size(), _stream()))
    res = {"idx": idx, "topk_length": tl}
    for name, t in (("logits", logits), ("softmax", sm), ("lse", lse)):
        if t is not None:
            res[name] = t
    return res


def indexer_scores(qi, ki, w, cu_seqlens, s_max: int, ld: int | None = None, out=None):
    """Dense indexer scores fp32 [T, ld] (columns >= s_max untouched)."""
    _need(qi, "qi", torch.bfloat16, 3)
    _need(ki, "ki", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hi, d = qi.shape
    ld = ld or (s_max + 3) // 4 * 4
    if out is None:
        out = torch.empty((T, ld), dtype=torch.float32, device=qi.device)
    _check("dsa_indexer_scores", lib().dsa_indexer_scores(_p(qi), _p(ki), _p(w), _p(cu_seqlens), cu_seqlens.numel() - 1,
                                                          T, Hi, d, s_max, _p(out), ld, _stream()))
    return out


def topk(scores, lengths, k: int, row_start=None, want_vals: bool = False, idx=None, topk_length=None):
    _need(scores, "scores", torch.float32, 2)
    _need(lengths, "lengths", torch.int32, 1)
    if row_start is not None:
        _need(row_start, "row_start", torch.int32, 1)
    T, ld = scores.shape
    dev = scores.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev) if idx is None else idx
    topk_length = torch.empty(T, dtype=torch.int32, device=dev) if topk_length is None else topk_length
    vals = torch.empty((T, k), dtype=torch.float32, device=dev) if want_vals else None
    _check("dsa_topk", lib().dsa_topk(_p(scores), ld, _p(lengths), _p(row_start), T, k, _p(idx), _p(topk_length),
                                      _p(vals), _stream()))
    return idx, topk_length, vals


def compact_sort_indices(indices, key_count: int, out=None):
    _need(indices, "indices", torch.int32, 2)
    T, K = indices.shape
    out = torch.empty_like(indices) if out is None else out
    lengths = torch.empty(T, dtype=torch.int32, device=indices.device)
    _check("dsa_compact_sort_indices", lib().dsa_compact_sort_indices(_p(indices), T, K, int(key_count), _p(out),
                                                                      _p(lengths), _stream()))
    return out, lengths


def indexer_topk_workspace_size(T: int, Hi: int, d: int, k: int, s_max: int) -> int:
    return int(lib().dsa_indexer_topk_workspace_size(T, Hi, d, k, s_max))


def indexer_topk(qi, ki, w, cu_seqlens, k: int, s_max: int, workspace=None, idx=None, topk_length=None):
    """Fused indexer + top-k: (idx [T, k] ascending global ids, topk_length [T])."""
    _need(qi, "qi", torch.bfloat16, 3)
    _need(ki, "ki", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hi, d = qi.shape
    dev = qi.device
    nbytes = indexer_topk_workspace_size(T, Hi, d, k, s_max)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev) if idx is None else idx
    topk_length = torch.empty(T, dtype=torch.int32, device=dev) if topk_length is None else topk_length
    _check("dsa_indexer_topk", lib().dsa_indexer_topk(_p(qi), _p(ki), _p(w), _p(cu_seqlens), cu_seqlens.numel() - 1,
                                                      T, Hi, d, k, s_max, _p(idx), _p(topk_length), _p(workspace),
                                                      workspace.numel() * workspace.element_size(), _stream()))
    return idx, topk_length


def indexer_topk_ex(qi, ki, w, cu_seqlens, k: int, s_max: int, want_softmax: bool = True, want_lse: bool = True,
                    workspace=None):
    """Fused indexer + top-k with its aligned logits, and optionally their
    softmax and lse: dict(idx, topk_length, logits[, softmax][, lse])."""
    _need(qi, "qi", torch.bfloat16, 3)
    _need(ki, "ki", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hi, d = qi.shape
    dev = qi.device
    if workspace is None:
        workspace = torch.empty(indexer_topk_workspace_size(T, Hi, d, k, s_max), dtype=torch.uint8, device=dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    tl = torch.empty(T, dtype=torch.int32, device=dev)
    logits = torch.empty((T, k), dtype=torch.float32, device=dev)
    sm = torch.empty((T, k), dtype=torch.float32, device=dev) if want_softmax else None
    lse = torch.empty(T, dtype=torch.float32, device=dev) if want_lse else None
    _check("dsa_indexer_topk_ex",
           lib().dsa_indexer_topk_ex(_p(qi), _p(ki), _p(w), _p(cu_seqlens), cu_seqlens.numel() - 1, T, Hi, d, k, s_max,
                                     _p(idx), _p(tl), _p(logits), _p(sm), _p(lse), _p(workspace),
                                     workspace.numel() * workspace.element_size(), _stream()))
    res = {"idx": idx, "topk_length": tl, "logits": logits}
    if sm is not None:
        res["softmax"] = sm
    if lse is not None:
        res["lse"] = lse
    return res


def topk_softmax(logits, idx, want_softmax: bool = True, want_lse: bool = True):
    """Softmax and lse of top-k logits over the slots with a valid id: (softmax or None, lse or None)."""
    _need(logits, "logits", torch.float32, 2)
    _need(idx, "idx", torch.int32, 2)
    T, k = logits.shape
    sm = torch.empty_like(logits) if want_softmax else None
    lse = torch.empty(T, dtype=torch.float32, device=logits.device) if want_lse else None
    _check("dsa_topk_softmax", lib().dsa_topk_softmax(_p(logits), _p(idx), T, k, _p(sm), _p(lse), _stream()))
    return sm, lse


class ForwardBuffers(ctypes.Structure):
    """dsa_forward_buffers (include/dsa.h), field for field."""
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "qi", "ki", "w", "cu_seqlens", "q", "kv", "sink", "qi_d", "ki_d", "w_d", "cu_seqlens_d", "q_d", "kv_d",
        "sink_d", "idx_d", "topk_length_d", "out_d", "lse_d", "workspace")] + [("ws_bytes", ctypes.c_size_t)] + [
        (name, ctypes.c_void_p) for name in ("idx", "topk_length", "out", "lse")]


def forward_host(host: dict, dev: dict, res_dev: dict, res_host: dict, workspace, n_docs: int, k: int, s_max: int,
                 scale: float, chunks: int = 4, copy_stream=None):
    """One forward step from host buffers through dsa_forward_host.

    host: qi, ki, w, cu_seqlens, q, kv, sink (page-locked CPU tensors; sink may
    be None); dev: device tensors of the same shapes; res_dev / res_host: idx,
    topk_length, out, lse on the device / in page-locked host memory.  Enqueues
    on the current stream and `copy_stream` and returns at once."""
    T, Hi, d = host["qi"].shape
    _, H, Dqk = host["q"].shape
    Dv = res_dev["out"].shape[2]
    if copy_stream is None:
        copy_stream = torch.cuda.Stream(device=dev["qi"].device)
    b = ForwardBuffers()
    for name in ("qi", "ki", "w", "cu_seqlens", "q", "kv", "sink"):
        setattr(b, name, None if host.get(name) is None else host[name].data_ptr())
        setattr(b, name + "_d", None if dev.get(name) is None else dev[name].data_ptr())
    for name in ("idx", "topk_length", "out", "lse"):
        setattr(b, name + "_d", res_dev[name].data_ptr())
        setattr(b, name, res_host[name].data_ptr())
    b.workspace = workspace.data_ptr()
    b.ws_bytes = workspace.numel() * workspace.element_size()
    _check("dsa_forward_host", lib().dsa_forward_host(ctypes.byref(b), n_docs, T, Hi, d, k, s_max, H, Dqk, Dv,
                                                      float(scale), chunks, _stream(),
                                                      ctypes.c_void_p(copy_stream.cuda_stream)))
    return copy_stream


def indexer_candidates(qi, ki, w, cu_seqlens, k: int, s_max: int, workspace=None):
    """Stage 1 of indexer_topk: fills and returns the candidate workspace."""
    _need(qi, "qi", torch.bfloat16, 3)
    _need(ki, "ki", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hi, d = qi.shape
    if workspace is None:
        workspace = torch.empty(indexer_topk_workspace_size(T, Hi, d, k, s_max), dtype=torch.uint8, device=qi.device)
    _check("dsa_indexer_candidates",
           lib().dsa_indexer_candidates(_p(qi), _p(ki), _p(w), _p(cu_seqlens), cu_seqlens.numel() - 1, T, Hi, d, k,
                                        s_max, _p(workspace), workspace.numel() * workspace.element_size(),
                                        _stream()))
    return workspace


def select_candidates(cu_seqlens, T: int, Hi: int, d: int, k: int, s_max: int, workspace, idx=None,
                      topk_length=None):
    """Stage 2 of indexer_topk over a workspace filled by indexer_candidates."""
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    _need(workspace, "workspace", torch.uint8, 1)
    dev = workspace.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev) if idx is None else idx
    topk_length = torch.empty(T, dtype=torch.int32, device=dev) if topk_length is None else topk_length
    _check("dsa_select_candidates",
           lib().dsa_select_candidates(_p(cu_seqlens), cu_seqlens.numel() - 1, T, Hi, d, k, s_max, _p(workspace),
                                       workspace.numel(), _p(idx), _p(topk_length), _stream()))
    return idx, topk_length


def indexer_topk_noalloc(qi, ki, w, cu_seqlens, k: int, s_max: int, idx=None, topk_length=None):
    """indexer_topk with the library's fixed scratch array (no workspace)."""
    _need(qi, "qi", torch.bfloat16, 3)
    _need(ki, "ki", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 2)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, Hi, d = qi.shape
    dev = qi.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev) if idx is None else idx
    topk_length = torch.empty(T, dtype=torch.int32, device=dev) if topk_length is None else topk_length
    _check("dsa_indexer_topk_noalloc",
           lib().dsa_indexer_topk_noalloc(_p(qi), _p(ki), _p(w), _p(cu_seqlens), cu_seqlens.numel() - 1, T, Hi, d,
                                          k, s_max, _p(idx), _p(topk_length), _stream()))
    return idx, topk_length


def sparse_attn_fwd(q, kv, idx, scale: float, topk_length=None, sink=None, v=None, want_lse_kv: bool = False,
                    want_max_logits: bool = False, out=None, lse=None, indexer_topk: int = 0):
    """Sparse MQA attention forward; returns dict(out, lse[, lse_kv][, max_logits][, lse_indexer]).
    indexer_topk > 0 adds lse_indexer (dsa_sparse_attn_fwd_ex)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(kv, "kv", torch.bfloat16, 2)
    _need(idx, "idx", torch.int32, 2)
    if topk_length is not None:
        _need(topk_length, "topk_length", torch.int32, 1)
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    if v is not None:
        _need(v, "v", torch.bfloat16, 2)
    T, H, Dqk = q.shape
    Tkv = kv.shape[0]
    Dv = v.shape[1] if v is not None else 512
    K = idx.shape[1]
    dev = q.device
    out = torch.empty((T, H, Dv), dtype=torch.bfloat16, device=dev) if out is None else out
    lse = torch.empty((T, H), dtype=torch.float32, device=dev) if lse is None else lse
    lse_kv = torch.empty((T, H), dtype=torch.float32, device=dev) if want_lse_kv else None
    ml = torch.empty((T, H), dtype=torch.float32, device=dev) if want_max_logits else None
    if indexer_topk:
        li = torch.empty((T, H), dtype=torch.float32, device=dev)
        _check("dsa_sparse_attn_fwd_ex",
               lib().dsa_sparse_attn_fwd_ex(_p(q), _p(kv), _p(v), _p(idx), _p(topk_length), _p(sink), T, Tkv, H, Dqk,
                                            Dv, K, float(scale), _p(out), _p(lse), _p(lse_kv), _p(ml),
                                            int(indexer_topk), _p(li), _stream()))
    else:
        li = None
        _check("dsa_sparse_attn_fwd",
               lib().dsa_sparse_attn_fwd(_p(q), _p(kv), _p(v), _p(idx), _p(topk_length), _p(sink), T, Tkv, H, Dqk,
                                         Dv, K, float(scale), _p(out), _p(lse), _p(lse_kv), _p(ml), _stream()))
    res = {"out": out, "lse": lse}
    if li is not None:
        res["lse_indexer"] = li
    if lse_kv is not None:
        res["lse_kv"] = lse_kv
    if ml is not None:
        res["max_logits"] = ml
    return res


def pack_routes(routes):
    _need(routes, "routes", torch.int32, 3)
    B, S, W = routes.shape
    Wp = (W + 3) // 4 * 4
    out = torch.empty((B * S, Wp), dtype=torch.int32, device=routes.device)
    _check("dsa_pack_routes", lib().dsa_pack_routes(_p(routes), B, S, W, _p(out), _stream()))
    return out


def sparse_attn_bwd_workspace_size(T: int, Tkv: int, H: int, K: int, deterministic: bool = True) -> int:
    return int(lib().dsa_sparse_attn_bwd_workspace_size_ex(T, Tkv, H, K, 1 if deterministic else 0))


def sparse_attn_bwd(q, kv, out, dout, lse_kv, idx, scale: float, topk_length=None, sink=None, workspace=None,
                    deterministic: bool = True):
    """Sparse attention backward (latent K = V): dict(dq bf16 [T, H, 576],
    dkv fp32 [Tkv, 576], d_sink fp32 [H] or None).  deterministic=False
    accumulates dkv with fp32 atomics (not bitwise reproducible)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(kv, "kv", torch.bfloat16, 2)
    _need(out, "out", torch.bfloat16, 3)
    _need(dout, "dout", torch.bfloat16, 3)
    _need(lse_kv, "lse_kv", torch.float32, 2)
    _need(idx, "idx", torch.int32, 2)
    if topk_length is not None:
        _need(topk_length, "topk_length", torch.int32, 1)
    if sink is not None:
        _need(sink, "sink", torch.float32, 1)
    T, H, Dqk = q.shape
    Tkv = kv.shape[0]
    Dv = out.shape[2]
    K = idx.shape[1]
    dev = q.device
    if workspace is None:
        workspace = torch.empty(sparse_attn_bwd_workspace_size(T, Tkv, H, K, deterministic), dtype=torch.uint8,
                                device=dev)
    dq = torch.empty((T, H, Dqk), dtype=torch.bfloat16, device=dev)
    dkv = torch.empty((Tkv, Dqk), dtype=torch.float32, device=dev)
    d_sink = torch.empty(H, dtype=torch.float32, device=dev) if sink is not None else None
    _check("dsa_sparse_attn_bwd_ex",
           lib().dsa_sparse_attn_bwd_ex(_p(q), _p(kv), _p(out), _p(dout), _p(lse_kv), _p(sink), _p(idx),
                                        _p(topk_length), T, Tkv, H, Dqk, Dv, K, float(scale), _p(dq), _p(dkv),
                                        _p(d_sink), 1 if deterministic else 0, _p(workspace),
                                        workspace.numel() * workspace.element_size(), _stream()))
    return {"dq": dq, "dkv": dkv, "d_sink": d_sink}


# The calls on the 8-bit cache are made once or twice per layer of a decode
# step, whose kernels run for a few microseconds.  Their arguments are checked
# by one condition each call; only when it fails are they looked at one by one
# for the error to raise.  Pointers and the stream go to ctypes as plain integers.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch.cuda.current_device
_Tensor, _U8, _I32, _F32, _BF16 = torch.Tensor, torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _ok(t, dtype, dim, device):
    """Whether t is a contiguous tensor of this kind on this device."""
    return (isinstance(t, _Tensor) and t.dtype == dtype and t.dim() == dim and t.is_contiguous() and
            t.get_device() == device)


# Sizes are 32-bit in the library, and ctypes takes larger ones modulo 2^32: the norm's, rotary's and the 4-bit
# cache's calls refuse them.
_MOST = 2 ** 31 - 1


def _need_size(t, name):
    if t.dim() > 1 and max(t.shape) > _MOST:
        raise ValueError(f"{name} is {list(t.shape)}: sizes are signed numbers of 32 bits")


def _refuse(device, *args):
    """Raises for the first of (tensor, name, dtype, dim, shape or None) that is not as it has to be."""
    for t, name, dtype, dim, shape in args:
        _need(t, name, dtype, dim)
        _need_size(t, name)
        if t.get_device() != device or device != _current_device():
            raise ValueError(f"{name} is on {t.device}: the tensors of a call are on the current device, "
                             f"cuda:{_current_device()}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError("inconsistent arguments")


def _kv8_refuse(cache, cache_scale, cu_seqlens, pos, block_table, rows, rows_name, T):
    _need(cache, "cache", _U8, 4)
    _need(cu_seqlens, "cu_seqlens", _I32, 1)
    n_blocks, _, heads, dim = cache.shape
    n_seqs = cu_seqlens.shape[0] - 1
    device = cache.get_device()
    args = [(cache, "cache", _U8, 4, None), (cache_scale, "cache_scale", _F32, 2, (n_blocks, heads)),
            (cu_seqlens, "cu_seqlens", _I32, 1, None)]
    if pos is not None:
        args.append((pos, "pos", _I32, 1, (n_seqs,)))
    if block_table is not None:
        _need(block_table, "block_table", _I32, 2)
        args.append((block_table, "block_table", _I32, 2, (n_seqs, block_table.shape[1])))
    _need(rows, rows_name, _BF16, 3)
    args.append((rows, rows_name, _BF16, 3, (rows.shape[0] if T is None else T, heads, dim)))
    _refuse(device, *args)


def kv8_write(src, cache, cache_scale, cu_seqlens, pos=None, block_table=None):
    """Quantises the bf16 rows src [T, Hc, D] into the E4M3 block cache (uint8
    [n_blocks, block, Hc, D], scale fp32 [n_blocks, Hc]), in place; returns both."""
    dev = cache.get_device() if isinstance(cache, _Tensor) else -1
    if not (dev >= 0 and dev == _current_device() and _ok(cache, _U8, 4, dev) and
            _ok(cache_scale, _F32, 2, dev) and _ok(cu_seqlens, _I32, 1, dev) and
            _ok(src, _BF16, 3, dev) and (pos is None or _ok(pos, _I32, 1, dev)) and
            (block_table is None or _ok(block_table, _I32, 2, dev))):
        _kv8_refuse(cache, cache_scale, cu_seqlens, pos, block_table, src, "src", None)
    n_blocks, block, heads, dim = cache.shape
    T = src.shape[0]
    n_seqs = cu_seqlens.shape[0] - 1
    rows, width = (n_seqs, 0) if block_table is None else block_table.shape
    if (src.shape != (T, heads, dim) or cache_scale.shape != (n_blocks, heads) or rows != n_seqs or
            (pos is not None and pos.shape[0] != n_seqs)):
        _kv8_refuse(cache, cache_scale, cu_seqlens, pos, block_table, src, "src", None)
    rc = (_lib or lib()).dsa_kv8_write(src.data_ptr(), cu_seqlens.data_ptr(), None if pos is None else pos.data_ptr(),
                                       None if block_table is None else block_table.data_ptr(), n_seqs, T, heads, dim,
                                       block, n_blocks, width, cache.data_ptr(), cache_scale.data_ptr(),
                                       _raw_stream(dev))
    if rc:
        _check("dsa_kv8_write", rc)
    return cache, cache_scale


def kv8_read(cache, cache_scale, cu_seqlens, T: int, pos=None, block_table=None, out=None):
    """Rows of the 8-bit block cache back to packed bf16 [T, Hc, D].  Rows behind the
    last sequence are not written: an `out` that is given keeps them, a new one has
    anything there."""
    dev = cache.get_device() if isinstance(cache, _Tensor) else -1
    if out is None and dev >= 0 and _ok(cache, _U8, 4, dev):
        out = torch.empty((T, cache.shape[2], cache.shape[3]), dtype=_BF16, device=cache.device)
    if not (dev >= 0 and dev == _current_device() and _ok(cache, _U8, 4, dev) and
            _ok(cache_scale, _F32, 2, dev) and _ok(cu_seqlens, _I32, 1, dev) and
            _ok(out, _BF16, 3, dev) and (pos is None or _ok(pos, _I32, 1, dev)) and
            (block_table is None or _ok(block_table, _I32, 2, dev))):
        _kv8_refuse(cache, cache_scale, cu_seqlens, pos, block_table, out, "out", T)
    n_blocks, block, heads, dim = cache.shape
    n_seqs = cu_seqlens.shape[0] - 1
    rows, width = (n_seqs, 0) if block_table is None else block_table.shape
    if (out.shape != (T, heads, dim) or cache_scale.shape != (n_blocks, heads) or rows != n_seqs or
            (pos is not None and pos.shape[0] != n_seqs)):
        _kv8_refuse(cache, cache_scale, cu_seqlens, pos, block_table, out, "out", T)
    rc = (_lib or lib()).dsa_kv8_read(cache.data_ptr(), cache_scale.data_ptr(), cu_seqlens.data_ptr(),
                                      None if pos is None else pos.data_ptr(),
                                      None if block_table is None else block_table.data_ptr(), n_seqs, T, heads, dim,
                                      block, n_blocks, width, out.data_ptr(), _raw_stream(dev))
    if rc:
        _check("dsa_kv8_read", rc)
    return out


def sparse_attn_fwd_kv8_workspace_size(T: int, H: int, Hc: int, Dqk: int, Dv: int, K: int) -> int:
    return int(lib().dsa_sparse_attn_fwd_kv8_workspace_size(T, H, Hc, Dqk, Dv, K))


def _attn_refuse(q, kv8, kv_scale, idx, topk_length, sink, v8, v_scale, cu_seqlens, block_table, out, lse, workspace):
    _need(q, "q", _BF16, 3)
    _need(kv8, "kv8", _U8, 4)
    T, H, Dqk = q.shape
    n_blocks, block, heads, _ = kv8.shape
    if (v8 is None) != (v_scale is None):
        raise ValueError("v8 and v_scale go together")
    if block_table is not None and cu_seqlens is None:
        raise ValueError("block_table needs cu_seqlens")
    args = [(q, "q", _BF16, 3, None), (kv8, "kv8", _U8, 4, (n_blocks, block, heads, Dqk)),
            (kv_scale, "kv_scale", _F32, 2, (n_blocks, heads))]
    _need(idx, "idx", _I32, 2)
    args.append((idx, "idx", _I32, 2, (T, idx.shape[1])))
    Dv = 512
    if v8 is not None:
        _need(v8, "v8", _U8, 4)
        Dv = v8.shape[3]
        args += [(v8, "v8", _U8, 4, (n_blocks, block, heads, Dv)), (v_scale, "v_scale", _F32, 2, (n_blocks, heads))]
    if block_table is not None:
        _need(block_table, "block_table", _I32, 2)
        args += [(block_table, "block_table", _I32, 2, None),
                 (cu_seqlens, "cu_seqlens", _I32, 1, (block_table.shape[0] + 1,))]
    args += [a for a in ((topk_length, "topk_length", _I32, 1, (T,)), (sink, "sink", _F32, 1, (H,)),
                         (out, "out", _BF16, 3, (T, H, Dv)), (lse, "lse", _F32, 2, (T, H)),
                         (workspace, "workspace", _U8, 1, None)) if a[0] is not None]
    _refuse(q.get_device(), *args)


def sparse_attn_fwd_kv8(q, kv8, kv_scale, idx, scale: float, topk_length=None, sink=None, v8=None, v_scale=None,
                        cu_seqlens=None, block_table=None, want_lse_kv: bool = False, want_max_logits: bool = False,
                        out=None, lse=None, workspace=None):
    """Sparse attention forward over the 8-bit block cache; returns dict(out, lse[, lse_kv][, max_logits]).
    idx holds cache rows, or, with block_table and cu_seqlens, positions in the row's sequence.  With a block_table,
    rows behind the last sequence are not written: tensors that are given keep them, new ones have anything there."""
    dev = q.get_device() if isinstance(q, _Tensor) else -1
    paged = block_table is not None
    if not (dev >= 0 and dev == _current_device() and _ok(q, _BF16, 3, dev) and _ok(kv8, _U8, 4, dev) and
            _ok(kv_scale, _F32, 2, dev) and
            _ok(idx, _I32, 2, dev) and (topk_length is None or _ok(topk_length, _I32, 1, dev)) and
            (sink is None or _ok(sink, _F32, 1, dev)) and
            (v8 is None if v_scale is None else _ok(v8, _U8, 4, dev) and _ok(v_scale, _F32, 2, dev)) and
            (not paged or _ok(block_table, _I32, 2, dev) and _ok(cu_seqlens, _I32, 1, dev)) and
            (out is None or _ok(out, _BF16, 3, dev)) and (lse is None or _ok(lse, _F32, 2, dev)) and
            (workspace is None or _ok(workspace, _U8, 1, dev))):
        _attn_refuse(q, kv8, kv_scale, idx, topk_length, sink, v8, v_scale, cu_seqlens, block_table, out, lse,
                     workspace)
    T, H, Dqk = q.shape
    n_blocks, block, heads, dim = kv8.shape
    K = idx.shape[1]
    Dv = 512 if v8 is None else v8.shape[3]
    n_seqs, width = (0, 0) if not paged else block_table.shape
    if (dim != Dqk or kv_scale.shape != (n_blocks, heads) or idx.shape[0] != T or
            (topk_length is not None and topk_length.shape[0] != T) or (sink is not None and sink.shape[0] != H) or
            (v8 is not None and (v8.shape != (n_blocks, block, heads, Dv) or v_scale.shape != (n_blocks, heads))) or
            (paged and cu_seqlens.shape[0] != n_seqs + 1) or (out is not None and out.shape != (T, H, Dv)) or
            (lse is not None and lse.shape != (T, H))):
        _attn_refuse(q, kv8, kv_scale, idx, topk_length, sink, v8, v_scale, cu_seqlens, block_table, out, lse,
                     workspace)
    device, empty = q.device, torch.empty
    if out is None:
        out = empty((T, H, Dv), dtype=_BF16, device=device)
    if lse is None:
        lse = empty((T, H), dtype=_F32, device=device)
    lse_kv = empty((T, H), dtype=_F32, device=device) if want_lse_kv else None
    ml = empty((T, H), dtype=_F32, device=device) if want_max_logits else None
    L = _lib or lib()
    if workspace is None:
        need = L.dsa_sparse_attn_fwd_kv8_workspace_size(T, H, heads, Dqk, Dv, K)
        if need:
            workspace = empty(need, dtype=_U8, device=device)
    rc = L.dsa_sparse_attn_fwd_kv8(
        q.data_ptr(), kv8.data_ptr(), kv_scale.data_ptr(), None if v8 is None else v8.data_ptr(),
        None if v8 is None else v_scale.data_ptr(), idx.data_ptr(),
        None if topk_length is None else topk_length.data_ptr(), None if sink is None else sink.data_ptr(),
        cu_seqlens.data_ptr() if paged else None, block_table.data_ptr() if paged else None, n_seqs, T, H, heads, Dqk,
        Dv, K, block, n_blocks, width, scale, out.data_ptr(), lse.data_ptr(),
        None if lse_kv is None else lse_kv.data_ptr(), None if ml is None else ml.data_ptr(),
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.shape[0],
        _raw_stream(dev))
    if rc:
        _check("dsa_sparse_attn_fwd_kv8", rc)
    res = {"out": out, "lse": lse}
    if lse_kv is not None:
        res["lse_kv"] = lse_kv
    if ml is not None:
        res["max_logits"] = ml
    return res


def _kv4_refuse(cache, cache_scale, cu_seqlens, pos, block_table, rows, rows_name, T):
    _need(cache, "cache", _U8, 4)
    _need(cu_seqlens, "cu_seqlens", _I32, 1)
    n_blocks, block, heads, half = cache.shape
    n_seqs = cu_seqlens.shape[0] - 1
    args = [(cache, "cache", _U8, 4, None), (cache_scale, "cache_scale", _U8, 4, (n_blocks, block, heads, half // 16)),
            (cu_seqlens, "cu_seqlens", _I32, 1, None)]
    if pos is not None:
        args.append((pos, "pos", _I32, 1, (n_seqs,)))
    if block_table is not None:
        _need(block_table, "block_table", _I32, 2)
        args.append((block_table, "block_table", _I32, 2, (n_seqs, block_table.shape[1])))
    _need(rows, rows_name, _BF16, 3)
    args.append((rows, rows_name, _BF16, 3, (rows.shape[0] if T is None else T, heads, 2 * half)))
    _refuse(cache.get_device(), *args)


def _kv4_call(rows, rows_name, T, cache, cache_scale, cu_seqlens, pos, block_table):
    """Checks what the writer and the reader share; their arguments from cu_seqlens to max_blocks."""
    p_ptr = t_ptr = width = 0
    try:
        n_blocks, block, heads, half = cache.shape
        n, dev = cu_seqlens.shape[0] - 1, cache.get_device()
        t, h, d = rows.shape
        ok = (cache.dtype is _U8 and dev == _get_device() and cache.is_contiguous() and cache_scale.dtype is _U8 and
              cache_scale.shape == (n_blocks, block, heads, half // 16) and cache_scale.is_contiguous() and
              cache_scale.get_device() == dev and cu_seqlens.dtype is _I32 and cu_seqlens.dim() == 1 and
              cu_seqlens.is_contiguous() and cu_seqlens.get_device() == dev and rows.dtype is _BF16 and h == heads and
              d == 2 * half and (T is None or t == T) and rows.is_contiguous() and rows.get_device() == dev and
              max(n_blocks, n, t) <= _MOST)
        if pos is not None:
            ok = ok and pos.dtype is _I32 and pos.shape == (n,) and pos.is_contiguous() and pos.get_device() == dev
            p_ptr = pos.data_ptr()
        if block_table is not None:
            m, width = block_table.shape
            ok = (ok and block_table.dtype is _I32 and m == n and block_table.is_contiguous() and
                  block_table.get_device() == dev and width <= _MOST)
            t_ptr = block_table.data_ptr()
    except (AttributeError, TypeError, ValueError, IndexError, RuntimeError):
        ok = False
    if not ok:
        _kv4_refuse(cache, cache_scale, cu_seqlens, pos, block_table, rows, rows_name, T)
    return (cu_seqlens.data_ptr(), p_ptr, t_ptr, n, t, heads, d, block, n_blocks, width), dev


def kv4_write(src, cache, cache_scale, cu_seqlens, pos=None, block_table=None):
    """Quantises the bf16 rows src [T, Hc, D] into the 4-bit block cache (codes uint8
    [n_blocks, block, Hc, D / 2], scale uint8 [n_blocks, block, Hc, D / 32]), in place; returns both."""
    args, dev = _kv4_call(src, "src", None, cache, cache_scale, cu_seqlens, pos, block_table)
    rc = (_lib or lib()).dsa_kv4_write(src.data_ptr(), *args, cache.data_ptr(), cache_scale.data_ptr(),
                                       _raw_stream(dev))
    if rc:
        _check("dsa_kv4_write", rc)
    return cache, cache_scale


def kv4_read(cache, cache_scale, cu_seqlens, T: int, pos=None, block_table=None, out=None):
    """Rows of the 4-bit block cache back to packed bf16 [T, Hc, D].  Rows behind the last
    sequence are not written: an `out` that is given keeps them, a new one has anything there."""
    if out is None and isinstance(cache, _Tensor) and cache.is_cuda and cache.dim() == 4:
        out = torch.empty((T, cache.shape[2], 2 * cache.shape[3]), dtype=_BF16, device=cache.device)
    args, dev = _kv4_call(out, "out", T, cache, cache_scale, cu_seqlens, pos, block_table)
    rc = (_lib or lib()).dsa_kv4_read(cache.data_ptr(), cache_scale.data_ptr(), *args, out.data_ptr(),
                                      _raw_stream(dev))
    if rc:
        _check("dsa_kv4_read", rc)
    return out


def sparse_attn_fwd_kv4_workspace_size(T: int, H: int, Hc: int, Dqk: int, Dv: int, K: int, block: int, n_blocks: int,
                                       paged: bool = False) -> int:
    return int(lib().dsa_sparse_attn_fwd_kv4_workspace_size(T, H, Hc, Dqk, Dv, K, block, n_blocks, 1 if paged else 0))


def _attn4_refuse(q, kv4, kv_scale, idx, topk_length, sink, v4, v_scale, cu_seqlens, block_table, out, lse, workspace):
    _need(q, "q", _BF16, 3)
    _need(kv4, "kv4", _U8, 4)
    T, H, Dqk = q.shape
    n_blocks, block, heads, _ = kv4.shape
    if (v4 is None) != (v_scale is None):
        raise ValueError("v4 and v_scale go together")
    if block_table is not None and cu_seqlens is None:
        raise ValueError("block_table needs cu_seqlens")
    args = [(q, "q", _BF16, 3, None), (kv4, "kv4", _U8, 4, (n_blocks, block, heads, Dqk // 2)),
            (kv_scale, "kv_scale", _U8, 4, (n_blocks, block, heads, Dqk // 32))]
    _need(idx, "idx", _I32, 2)
    args.append((idx, "idx", _I32, 2, (T, idx.shape[1])))
    Dv = 512
    if v4 is not None:
        _need(v4, "v4", _U8, 4)
        Dv = 2 * v4.shape[3]
        args += [(v4, "v4", _U8, 4, (n_blocks, block, heads, Dv // 2)),
                 (v_scale, "v_scale", _U8, 4, (n_blocks, block, heads, Dv // 32))]
    if block_table is not None:
        _need(block_table, "block_table", _I32, 2)
        args += [(block_table, "block_table", _I32, 2, None),
                 (cu_seqlens, "cu_seqlens", _I32, 1, (block_table.shape[0] + 1,))]
    args += [a for a in ((topk_length, "topk_length", _I32, 1, (T,)), (sink, "sink", _F32, 1, (H,)),
                         (out, "out", _BF16, 3, (T, H, Dv)), (lse, "lse", _F32, 2, (T, H)),
                         (workspace, "workspace", _U8, 1, None)) if a[0] is not None]
    _refuse(q.get_device(), *args)


def sparse_attn_fwd_kv4(q, kv4, kv_scale, idx, scale: float, topk_length=None, sink=None, v4=None, v_scale=None,
                        cu_seqlens=None, block_table=None, want_lse_kv: bool = False, want_max_logits: bool = False,
                        out=None, lse=None, workspace=None):
    """Sparse attention forward over the 4-bit block cache; returns dict(out, lse[, lse_kv][, max_logits]).
    idx, block_table and rows behind the last sequence as in sparse_attn_fwd_kv8."""
    l_ptr = z_ptr = v_ptr = vs_ptr = c_ptr = t_ptr = n_seqs = width = w_ptr = w_bytes = 0
    Dv = 512
    try:
        T, H, Dqk = q.shape
        n_blocks, block, heads, half = kv4.shape
        dev, (rows, K) = q.get_device(), idx.shape
        ok = (q.dtype is _BF16 and dev == _get_device() and q.is_contiguous() and kv4.dtype is _U8 and
              2 * half == Dqk and kv4.is_contiguous() and kv4.get_device() == dev and kv_scale.dtype is _U8 and
              kv_scale.shape == (n_blocks, block, heads, half // 16) and kv_scale.is_contiguous() and
              kv_scale.get_device() == dev and idx.dtype is _I32 and rows == T and idx.is_contiguous() and
              idx.get_device() == dev and max(T, K, n_blocks) <= _MOST)
        if topk_length is not None:
            ok = (ok and topk_length.dtype is _I32 and topk_length.shape == (T,) and topk_length.is_contiguous() and
                  topk_length.get_device() == dev)
            l_ptr = topk_length.data_ptr()
        if sink is not None:
            ok = (ok and sink.dtype is _F32 and sink.shape == (H,) and sink.is_contiguous() and
                  sink.get_device() == dev)
            z_ptr = sink.data_ptr()
        if v4 is not None:
            half = v4.shape[3]
            Dv = 2 * half
            ok = (ok and v4.dtype is _U8 and v4.shape == (n_blocks, block, heads, half) and v4.is_contiguous() and
                  v4.get_device() == dev and v_scale.dtype is _U8 and
                  v_scale.shape == (n_blocks, block, heads, half // 16) and v_scale.is_contiguous() and
                  v_scale.get_device() == dev)
            v_ptr, vs_ptr = v4.data_ptr(), v_scale.data_ptr()
        elif v_scale is not None:
            ok = False
        if block_table is not None:
            n_seqs, width = block_table.shape
            ok = (ok and block_table.dtype is _I32 and block_table.is_contiguous() and
                  block_table.get_device() == dev and cu_seqlens.dtype is _I32 and cu_seqlens.shape == (n_seqs + 1,) and
                  cu_seqlens.is_contiguous() and cu_seqlens.get_device() == dev and max(n_seqs, width) <= _MOST)
            t_ptr, c_ptr = block_table.data_ptr(), cu_seqlens.data_ptr()
        if out is not None:
            ok = (ok and out.dtype is _BF16 and out.shape == (T, H, Dv) and out.is_contiguous() and
                  out.get_device() == dev)
        if lse is not None:
            ok = ok and lse.dtype is _F32 and lse.shape == (T, H) and lse.is_contiguous() and lse.get_device() == dev
        ok = ok and (workspace is None or _ok(workspace, _U8, 1, dev))
    except (AttributeError, TypeError, ValueError, IndexError, RuntimeError):
        ok = False
    if not ok:
        _attn4_refuse(q, kv4, kv_scale, idx, topk_length, sink, v4, v_scale, cu_seqlens, block_table, out, lse,
                      workspace)
    device, empty = q.device, torch.empty
    res = {}
    if out is None:
        out = empty((T, H, Dv), dtype=_BF16, device=device)
    if lse is None:
        lse = empty((T, H), dtype=_F32, device=device)
    res["out"], res["lse"] = out, lse
    k_ptr = m_ptr = 0
    if want_lse_kv:
        res["lse_kv"] = lse_kv = empty((T, H), dtype=_F32, device=device)
        k_ptr = lse_kv.data_ptr()
    if want_max_logits:
        res["max_logits"] = ml = empty((T, H), dtype=_F32, device=device)
        m_ptr = ml.data_ptr()
    L = _lib or lib()
    if workspace is None:
        need = L.dsa_sparse_attn_fwd_kv4_workspace_size(T, H, heads, Dqk, Dv, K, block, n_blocks, 1 if t_ptr else 0)
        if need:
            workspace = empty((need,), dtype=_U8, device=device)
    if workspace is not None:
        w_ptr, w_bytes = workspace.data_ptr(), workspace.shape[0]
    rc = L.dsa_sparse_attn_fwd_kv4(q.data_ptr(), kv4.data_ptr(), kv_scale.data_ptr(), v_ptr, vs_ptr, idx.data_ptr(), l_ptr,
                                   z_ptr, c_ptr, t_ptr, n_seqs, T, H, heads, Dqk, Dv, K, block, n_blocks, width, scale,
                                   out.data_ptr(), lse.data_ptr(), k_ptr, m_ptr, w_ptr, w_bytes, _raw_stream(dev))
    if rc:
        _check("dsa_sparse_attn_fwd_kv4", rc)
    return res


# Norm and rotary positions: rows may lie apart, so what is asked of a tensor is
# a last dimension without gaps; the C side checks the other strides.  As above, one
# condition a call, and a look at each argument only when it fails (or when one is no tensor).
_NORM_FORMS = {"bf16": (0, 0), "e4m3": (1, 128), "mxfp8": (2, 32)}
_F64 = torch.float64
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _strided_refuse(device, *args):
    """Raises for the first of (tensor, name, dtype, shape, strided) that is not as it has to be."""
    for t, name, dtype, shape, strided in args:
        if not isinstance(t, _Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        _need_size(t, name)
        if t.get_device() != device or device != _current_device():
            raise ValueError(f"{name} is on {t.device}: the tensors of a call are on the current device, "
                             f"cuda:{_current_device()}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not (t.stride(-1) == 1 if strided else t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous" + (" in its last dimension" if strided else ""))
    raise ValueError("inconsistent arguments")


def _need_dim(t, name, dim):
    if not isinstance(t, _Tensor) or t.dim() != dim:
        raise TypeError(f"{name} must be a torch.Tensor of {dim} dimensions")
    return t


def _norm_refuse(x, weight, residual, fmt, out, sum_out, scale):
    if fmt not in _NORM_FORMS:
        raise ValueError(f"fmt must be one of {sorted(_NORM_FORMS)}, got {fmt!r}")
    T, D = shape = _need_dim(x, "x", 2).shape
    form, group = _NORM_FORMS[fmt]
    if scale is not None and not form:
        raise ValueError("scale goes with the 8-bit forms")
    _strided_refuse(x.get_device(), (x, "x", _BF16, shape, True), (weight, "weight", _F32, (D,), False),
                    *[a for a in ((residual, "residual", _BF16, shape, True),
                                  (out, "out", _U8 if form else _BF16, shape, True),
                                  (sum_out, "sum_out", _BF16, shape, True),
                                  (scale, "scale", _F32 if form == 1 else _U8, (T, D // group if form else 0), False))
                      if a[0] is not None])


def rms_norm_fwd(x, weight, eps: float, residual=None, fmt: str = "bf16", out=None, sum_out=None, scale=None,
                 want_rstd: bool = False):
    """Root-mean-square norm of the rows of x [T, D] (plus residual): dict(out[, sum][, scale][, rstd]).
    fmt "bf16": out bf16; "e4m3": out uint8 codes and scale fp32 [T, D / 128]; "mxfp8": codes and
    scale uint8 [T, D / 32] (E8M0).  sum: x + residual in bf16, with a residual.  Rows of x, residual, out and
    sum_out may lie apart; out and sum_out may be x or residual."""
    try:
        form, group = _NORM_FORMS[fmt]
        T, D = shape = x.shape
        dev, xs = x.get_device(), x.stride()
        ok = (x.dtype is _BF16 and xs[1] == 1 and dev == _get_device() and weight.dtype is _F32 and
              weight.shape == (D,) and weight.stride(0) == 1 and weight.get_device() == dev and max(T, D) <= _MOST)
        r_ptr = r_ld = y_ptr = s_ptr = c_ptr = 0
        if residual is not None:
            st = residual.stride()
            ok = (ok and residual.dtype is _BF16 and residual.shape == shape and st[1] == 1 and
                  residual.get_device() == dev)
            r_ptr, r_ld = residual.data_ptr(), st[0]
        y_ld = s_ld = D
        if out is not None:
            st = out.stride()
            ok = (ok and out.dtype is (_U8 if form else _BF16) and out.shape == shape and st[1] == 1 and
                  out.get_device() == dev)
            y_ld = st[0]
        if sum_out is not None:
            st = sum_out.stride()
            ok = (ok and sum_out.dtype is _BF16 and sum_out.shape == shape and st[1] == 1 and
                  sum_out.get_device() == dev)
            s_ld = st[0]
        if scale is not None:
            ok = (ok and form and scale.dtype is (_F32 if form == 1 else _U8) and scale.shape == (T, D // group) and
                  scale.is_contiguous() and scale.get_device() == dev)
    except (AttributeError, KeyError, TypeError, ValueError, IndexError, RuntimeError):
        ok = False
    if not ok:
        _norm_refuse(x, weight, residual, fmt, out, sum_out, scale)
    empty, device = torch.empty, x.device
    res = {}
    if out is None:
        out = empty(shape, dtype=_U8 if form else _BF16, device=device)
    res["out"], y_ptr = out, out.data_ptr()
    if sum_out is None and residual is not None:
        sum_out = empty(shape, dtype=_BF16, device=device)
    if sum_out is not None:
        res["sum"], s_ptr = sum_out, sum_out.data_ptr()
    if form:
        if scale is None:
            scale = empty((T, D // group), dtype=_F32 if form == 1 else _U8, device=device)
        res["scale"], c_ptr = scale, scale.data_ptr()
    rstd_ptr = 0
    if want_rstd:
        res["rstd"] = rstd = empty((T,), dtype=_F32, device=device)
        rstd_ptr = rstd.data_ptr()
    if T <= 1:  # a row's stride to the next is nobody's business
        x_ld = r_ld = y_ld = s_ld = D
    else:
        x_ld = xs[0]
    rc = (_lib or lib()).dsa_rms_norm_fwd(x.data_ptr(), x_ld, r_ptr, r_ld, weight.data_ptr(), T, D, eps, form, y_ptr,
                                          y_ld, c_ptr, s_ptr, s_ld, rstd_ptr, _raw_stream(dev))
    if rc:
        _check("dsa_rms_norm_fwd", rc)
    return res


def rms_norm_bwd_workspace_size(T: int, D: int) -> int:
    return int(lib().dsa_rms_norm_bwd_workspace_size(T, D))


def rms_norm_bwd(dy, x, weight, rstd, d_sum=None, want_dweight: bool = True, dx=None, workspace=None):
    """Backward of rms_norm_fwd: dict(dx bf16 [T, D], dweight fp32 [D] or None).  x: the forward's sum (its x
    without a residual); dx is the gradient of x and of the residual alike.  Rows may lie apart."""
    try:
        T, D = shape = x.shape
        dev, xs, ys = x.get_device(), x.stride(), dy.stride()
        ok = (x.dtype is _BF16 and xs[1] == 1 and dev == _get_device() and dy.dtype is _BF16 and dy.shape == shape and
              ys[1] == 1 and dy.get_device() == dev and weight.dtype is _F32 and weight.shape == (D,) and
              weight.stride(0) == 1 and weight.get_device() == dev and rstd.dtype is _F32 and rstd.shape == (T,) and
              rstd.is_contiguous() and rstd.get_device() == dev and max(T, D) <= _MOST)
        x_ld, y_ld, s_ptr, s_ld, o_ld = xs[0], ys[0], 0, 0, D
        if d_sum is not None:
            st = d_sum.stride()
            ok = ok and d_sum.dtype is _BF16 and d_sum.shape == shape and st[1] == 1 and d_sum.get_device() == dev
            s_ptr, s_ld = d_sum.data_ptr(), st[0]
        if dx is not None:
            st = dx.stride()
            ok = ok and dx.dtype is _BF16 and dx.shape == shape and st[1] == 1 and dx.get_device() == dev
            o_ld = st[0]
        ok = ok and (workspace is None or _ok(workspace, _U8, 1, dev))
    except (AttributeError, TypeError, ValueError, IndexError, RuntimeError):
        ok = False
    if not ok:
        T, D = shape = _need_dim(x, "x", 2).shape
        args = [(dy, "dy", _BF16, shape, True), (x, "x", _BF16, shape, True), (weight, "weight", _F32, (D,), False),
                (rstd, "rstd", _F32, (T,), False)]
        args += [a for a in ((d_sum, "d_sum", _BF16, shape, True), (dx, "dx", _BF16, shape, True)) if a[0] is not None]
        if workspace is not None:
            args.append((workspace, "workspace", _U8, (workspace.numel(),) if isinstance(workspace, _Tensor) else (), False))
        _strided_refuse(x.get_device(), *args)
    empty, device = torch.empty, x.device
    if dx is None:
        dx = empty(shape, dtype=_BF16, device=device)
    if T <= 1:  # a row's stride to the next is nobody's business
        x_ld = y_ld = s_ld = o_ld = D
    L = _lib or lib()
    dweight, w_ptr, ws_ptr, ws_bytes = None, 0, 0, 0
    if want_dweight:
        dweight = empty((D,), dtype=_F32, device=device)
        w_ptr = dweight.data_ptr()
        if workspace is None:
            workspace = empty((L.dsa_rms_norm_bwd_workspace_size(T, D),), dtype=_U8, device=device)
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.shape[0]
    rc = L.dsa_rms_norm_bwd(dy.data_ptr(), y_ld, x.data_ptr(), x_ld, weight.data_ptr(), rstd.data_ptr(), s_ptr, s_ld, T, D,
                            dx.data_ptr(), o_ld, w_ptr, ws_ptr, ws_bytes, _raw_stream(dev))
    if rc:
        _check("dsa_rms_norm_bwd", rc)
    return {"dx": dx, "dweight": dweight}


_ROTARY_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rotary_inv_freq(R: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, first: int = 4096,
                    beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(inv_freq fp64 [R / 2] on `device`, mul) for rotary(); scaling "plain", "linear", "ntk" or "yarn"."""
    if scaling not in _ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY_SCALINGS)}, got {scaling!r}")
    freq, mul = torch.empty(max(R, 0) // 2, dtype=torch.float64), ctypes.c_float(0.0)
    _check("dsa_rotary_inv_freq",
           lib().dsa_rotary_inv_freq(R, base, _ROTARY_SCALINGS[scaling], factor, first, beta_fast, beta_slow,
                                     freq.data_ptr(), ctypes.byref(mul)))
    return freq.to(device or "cuda"), float(mul.value)


def _rotary_refuse(x, inv_freq, cu_seqlens, pos, x2, out, out2):
    T, _, R = shape = _need_dim(x, "x", 3).shape
    if x2 is None and out2 is not None:
        raise ValueError("out2 goes with x2")
    shape2 = () if x2 is None else (T, _need_dim(x2, "x2", 3).shape[1], R)
    _need(cu_seqlens, "cu_seqlens", _I32, 1)
    args = [(x, "x", _BF16, shape, True), (inv_freq, "inv_freq", _F64, (R // 2,), False),
            (cu_seqlens, "cu_seqlens", _I32, cu_seqlens.shape, False)]
    args += [a for a in ((pos, "pos", _I32, (cu_seqlens.shape[0] - 1,), False), (x2, "x2", _BF16, shape2, True),
                         (out, "out", _BF16, shape, True), (out2, "out2", _BF16, shape2, True)) if a[0] is not None]
    _strided_refuse(x.get_device(), *args)


def rotary(x, inv_freq, cu_seqlens, pos=None, x2=None, interleaved: bool = True, mul: float = 1.0,
           inverse: bool = False, out=None, out2=None):
    """Rotary positions of x bf16 [T, H, R] and, in the same call, x2 [T, H2, R]: (out, out2 or None).  Token t of
    sequence b stands at pos[b] + t - cu_seqlens[b] (pos None: 0).  Part of a head is x[..., a:b], in place with out=x;
    inverse: the adjoint, for gradients.  Rows of tokens outside the sequences are not written."""
    H2 = a2 = b2 = c2 = d2 = x2_ptr = y2_ptr = p_ptr = 0
    try:
        T, H, R = shape = x.shape
        dev = x.get_device()
        a1, b1, last = x.stride()
        n = cu_seqlens.shape[0] - 1
        ok = (x.dtype is _BF16 and last == 1 and dev == _get_device() and inv_freq.dtype is _F64 and
              inv_freq.shape == (R // 2,) and inv_freq.is_contiguous() and inv_freq.get_device() == dev and
              cu_seqlens.dtype is _I32 and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous() and
              cu_seqlens.get_device() == dev and max(T, H, R, n) <= _MOST)
        if pos is not None:
            ok = ok and pos.dtype is _I32 and pos.shape == (n,) and pos.is_contiguous() and pos.get_device() == dev
            p_ptr = pos.data_ptr()
        c1, d1 = H * R, R
        if out is not None:
            c1, d1, last = out.stride()
            ok = ok and out.dtype is _BF16 and out.shape == shape and last == 1 and out.get_device() == dev
        if x2 is not None:
            t2, H2, r2 = shape2 = x2.shape
            a2, b2, last = x2.stride()
            ok = ok and x2.dtype is _BF16 and t2 == T and r2 == R and last == 1 and x2.get_device() == dev and H2 <= _MOST
            x2_ptr = x2.data_ptr()
            c2, d2 = H2 * R, R
            if out2 is not None:
                c2, d2, last = out2.stride()
                ok = ok and out2.dtype is _BF16 and out2.shape == shape2 and last == 1 and out2.get_device() == dev
        elif out2 is not None:
            ok = False
    except (AttributeError, TypeError, ValueError, IndexError, RuntimeError):
        ok = False
    if not ok:
        _rotary_refuse(x, inv_freq, cu_seqlens, pos, x2, out, out2)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=x.device)
    if x2 is not None:
        if out2 is None:
            out2 = torch.empty(shape2, dtype=_BF16, device=x.device)
        y2_ptr = out2.data_ptr()
    if T <= 1:  # strides of a single token or head are nobody's business
        a1, c1, a2, c2 = H * R, H * R, H2 * R, H2 * R
    if H == 1:
        b1 = d1 = R
    if H2 == 1:
        b2 = d2 = R
    rc = (_lib or lib()).dsa_rotary(x.data_ptr(), a1, b1, H, x2_ptr, a2, b2, H2, inv_freq.data_ptr(),
                                    cu_seqlens.data_ptr(), p_ptr, n, T, R, 1 if interleaved else 0, 1 if inverse else 0,
                                    mul, out.data_ptr(), c1, d1, y2_ptr, c2, d2, _raw_stream(dev))
    if rc:
        _check("dsa_rotary", rc)
    return out, out2
