"""Exact scaled-dot-product attention on GB300: Python binding of ``libbwattn``.

Every function here only checks and marshals arguments (shapes, dtypes, device pointers,
the current CUDA stream) and calls the C-ABI in ``libbwattn.so``; all arithmetic runs in the
library's CUDA kernels. PyTorch supplies device memory and streams. There is no fallback:
if the library is missing or a call fails, a ``RuntimeError`` is raised.

Calls (see ``include/bwattn.h`` for the full contract):

* ``attn_fwd(q, k, v, causal, scale, window=0)``: prefill / cross attention, q [B, Hq, Nq, d],
  k, v [B, Hkv, Nk, d]; bf16 (tcgen05 kernel) or fp32 (fp32 FMA kernel); ``window`` > 0 adds a
  causal sliding window.
* ``attn_fwd_host(...)``: the same prefill from host tensors, with the copies overlapping the
  kernels (workspace from ``fwd_host_workspace_size``).
* ``attn_decode(q, kcache, vcache, nk, num_splits)``: single-query split-K decode,
  q [B, Hq, d], caches [B, Hkv, cap, d] bf16, nk [B] int32 on the device;
  ``attn_decode_paged`` over a paged cache and a block table; ``attn_decode_fp8`` /
  ``attn_decode_paged_fp8`` over E4M3 caches with per-channel scales.
* ``attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal)``:
  packed sequences, q [total_q, Hq, d], k, v [total_k, Hkv, d] bf16.
* Speculative decoding: ``attn_tree`` / ``attn_tree_paged`` (drafted token trees over a cache),
  ``attn_tree_mask`` (their masks and positions from parent links), ``kv_plan_paged`` (block tables
  and slots from request lengths), ``kv_append_paged`` / ``kv_append_paged_fp8`` (new K/V rows into
  the pages).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

__all__ = [
    "attn_fwd", "attn_fwd_host", "attn_decode", "attn_decode_paged", "attn_decode_fp8", "attn_decode_paged_fp8",
    "attn_varlen", "attn_tree", "attn_tree_paged", "attn_tree_mask", "kv_plan_paged", "kv_append_paged",
    "kv_append_paged_fp8", "fwd_host_workspace_size", "decode_workspace_size", "varlen_workspace_size",
    "tree_workspace_size",
    "get_status", "clear_status", "set_wait_timeout_ns", "test_wait_timeout", "launch_count", "lib",
    "status_string", "BwattnError", "OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_CUDA", "ERR_TIMEOUT",
]

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, 1, 2, 3, 4
DTYPE_FP32, DTYPE_BF16 = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbwattn.so")
_lock = threading.Lock()
_lib = None


class BwattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libbwattn.so not found at {LIB_PATH}; build it with "
                "`python -m exact_attention_flashattn_gb300.build` (needs nvcc for sm_103a)")
        L = ctypes.CDLL(LIB_PATH)
        vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.attn_fwd.argtypes = [vp, vp, vp, vp, vp] + [ci] * 7 + [cf, ci, vp]
        L.attn_fwd.restype = ci
        L.attn_fwd_window.argtypes = [vp, vp, vp, vp, vp] + [ci] * 7 + [cf, ci, vp]
        L.attn_fwd_window.restype = ci
        L.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp] + [ci] * 7 + [cf, ci, vp, sz, vp]
        L.attn_fwd_host.restype = ci
        L.attn_fwd_host_workspace_size.argtypes = [ci] * 7
        L.attn_fwd_host_workspace_size.restype = sz
        L.attn_decode_workspace_size.argtypes = [ci, ci, ci, ci]
        L.attn_decode_workspace_size.restype = sz
        L.attn_decode.argtypes = [vp, vp, vp, vp, vp] + [ci] * 6 + [cf, vp, vp, sz, vp]
        L.attn_decode.restype = ci
        L.attn_decode_paged.argtypes = [vp] * 6 + [ci] * 8 + [cf, vp, vp, sz, vp]
        L.attn_decode_fp8.argtypes = [vp] * 7 + [ci] * 6 + [cf, vp, vp, sz, vp]
        L.attn_decode_paged_fp8.argtypes = [vp] * 8 + [ci] * 8 + [cf, vp, vp, sz, vp]
        L.attn_decode_paged.restype = ci
        L.attn_varlen_workspace_size.argtypes = [ci] * 5
        L.attn_varlen_workspace_size.restype = sz
        L.attn_varlen.argtypes = [vp] * 7 + [ci] * 9 + [cf, vp, sz, vp]
        L.attn_varlen.restype = ci
        L.attn_varlen_window.argtypes = [vp] * 7 + [ci] * 9 + [cf, vp, sz, vp]
        L.attn_varlen_window.restype = ci
        i64 = ctypes.c_int64
        L.attn_tree_workspace_size.argtypes = [ci] * 5
        L.attn_tree_workspace_size.restype = sz
        L.attn_tree.argtypes = [vp] * 10 + [ci] * 7 + [i64] * 3 + [cf, vp, sz, vp]
        L.attn_tree.restype = ci
        L.attn_tree_paged.argtypes = [vp] * 11 + [ci] * 9 + [i64] * 3 + [cf, vp, sz, vp]
        L.attn_tree_paged.restype = ci
        L.attn_tree_mask.argtypes = [vp] * 5 + [ci] * 3 + [vp]
        L.attn_tree_mask.restype = ci
        L.kv_plan_paged.argtypes = [vp] * 11 + [ci] * 5 + [vp]
        L.kv_plan_paged.restype = ci
        L.kv_append_paged.argtypes = [vp] * 6 + [ci] * 6 + [i64] * 2 + [vp]
        L.kv_append_paged.restype = ci
        L.kv_append_paged_fp8.argtypes = [vp] * 8 + [ci] * 6 + [i64] * 2 + [vp]
        L.kv_append_paged_fp8.restype = ci
        L.bwattn_last_cuda_error.argtypes = []
        L.bwattn_last_cuda_error.restype = ci
        L.bwattn_status_string.argtypes = [ci]
        L.bwattn_status_string.restype = ctypes.c_char_p
        L.bwattn_get_status.argtypes = [vp]
        L.bwattn_get_status.restype = ci
        L.bwattn_clear_status.argtypes = [vp]
        L.bwattn_clear_status.restype = ci
        L.bwattn_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
        L.bwattn_set_wait_timeout_ns.restype = None
        L.bwattn_test_wait_timeout.argtypes = [vp]
        L.bwattn_test_wait_timeout.restype = ci
        L.bwattn_launch_count.argtypes = []
        L.bwattn_launch_count.restype = ctypes.c_uint64
        L.bwattn_version.argtypes = []
        L.bwattn_version.restype = ci
        _lib = L
        return L


def status_string(status: int) -> str:
    try:
        return lib().bwattn_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - only when the library itself is missing
        return "unknown"


def _check(rc: int, what: str):
    if rc != OK:
        if rc == ERR_CUDA:
            err = lib().bwattn_last_cuda_error()
            raise BwattnError(rc, f"{what} (cudaError {err})")
        raise BwattnError(rc, what)


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _cuda(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _scale(scale, d):
    return (1.0 / math.sqrt(d)) if scale is None else float(scale)


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = True, scale: float | None = None,
             out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = True, stream=None, window: int = 0):
    """Prefill / cross attention. q [B, Hq, Nq, d]; k, v [B, Hkv, Nk, d] -> (o, lse or None).

    ``window`` > 0 (causal only): sliding window of that many keys ending at each query's limit."""
    if window and not causal:
        raise ValueError("a sliding window needs causal=True")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, N, d]")
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if Bk != B or dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, Hkv, Nk, d] with q's B and d")
    if q.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif q.dtype == torch.float32:
        dt = DTYPE_FP32
    else:
        raise ValueError(f"unsupported dtype {q.dtype}")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _cuda(t, n, q.dtype)
    if out is None:
        out = torch.empty_like(q)
    _cuda(out, "out", q.dtype)
    lse_t = None
    if lse is True:
        lse_t = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    elif isinstance(lse, torch.Tensor):
        lse_t = lse
        _cuda(lse_t, "lse", torch.float32)
    if window:
        rc = lib().attn_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse_t), B, Hq, Hkv, Nq, Nk, d,
                                   int(window), _scale(scale, d), dt, _stream(stream))
        _check(rc, "attn_fwd_window")
        return out, lse_t
    rc = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse_t), B, Hq, Hkv, Nq, Nk, d, int(bool(causal)),
                        _scale(scale, d), dt, _stream(stream))
    _check(rc, "attn_fwd")
    return out, lse_t


def fwd_host_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int, dtype=torch.bfloat16) -> int:
    dt = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_FP32
    return int(lib().attn_fwd_host_workspace_size(B, Hq, Hkv, Nq, Nk, d, dt))


def attn_fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = True, scale: float | None = None,
                  out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = True,
                  workspace: torch.Tensor | None = None, stream=None, device=None):
    """attn_fwd on host (CPU) tensors, copies included; pinned memory lets them overlap the kernels.
    The call is asynchronous on ``stream`` (the current stream of ``device`` by default): read
    ``out`` after synchronising it."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor")
    if q.dim() != 4 or k.dim() != 4 or tuple(v.shape) != tuple(k.shape):
        raise ValueError("q [B, Hq, Nq, d]; k, v [B, Hkv, Nk, d]")
    B, Hq, Nq, d = q.shape
    _, Hkv, Nk, _ = k.shape
    if q.dtype not in (torch.bfloat16, torch.float32) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must all be bf16 or all fp32")
    dt = DTYPE_BF16 if q.dtype == torch.bfloat16 else DTYPE_FP32
    if out is None:
        out = torch.empty_like(q, pin_memory=q.is_pinned())
    if out.is_cuda or out.dtype != q.dtype or tuple(out.shape) != tuple(q.shape) or not out.is_contiguous():
        raise ValueError("out must be a contiguous host tensor like q")
    lse_t = None
    if lse is True:
        lse_t = torch.empty((B, Hq, Nq), dtype=torch.float32, pin_memory=q.is_pinned())
    elif isinstance(lse, torch.Tensor):
        lse_t = lse
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    need = int(lib().attn_fwd_host_workspace_size(B, Hq, Hkv, Nq, Nk, d, dt))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _cuda(workspace, "workspace")
    with torch.cuda.device(dev):
        rc = lib().attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse_t), B, Hq, Hkv, Nq, Nk, d,
                                 int(bool(causal)), _scale(scale, d), dt, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "attn_fwd_host")
    return out, lse_t


def decode_workspace_size(B: int, Hq: int, d: int, num_splits: int) -> int:
    return int(lib().attn_decode_workspace_size(B, Hq, d, num_splits))


def attn_decode(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, nk: torch.Tensor, num_splits: int,
                scale: float | None = None, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                lse: torch.Tensor | bool | None = True, stream=None):
    """Single-query decode. q [B, Hq, d]; caches [B, Hkv, cap, d]; nk [B] int32 (device)."""
    if q.dim() != 3 or kcache.dim() != 4:
        raise ValueError("q must be [B, Hq, d] and caches [B, Hkv, cap, d]")
    B, Hq, d = q.shape
    Bk, Hkv, cap, dk = kcache.shape
    if Bk != B or dk != d or tuple(vcache.shape) != tuple(kcache.shape):
        raise ValueError("kcache and vcache must be [B, Hkv, cap, d] with q's B and d")
    for t, n in ((q, "q"), (kcache, "kcache"), (vcache, "vcache")):
        _cuda(t, n, torch.bfloat16)
    _cuda(nk, "nk", torch.int32)
    if out is None:
        out = torch.empty_like(q)
    _cuda(out, "out", torch.bfloat16)
    lse_t = None
    if lse is True:
        lse_t = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    elif isinstance(lse, torch.Tensor):
        lse_t = lse
        _cuda(lse_t, "lse", torch.float32)
    need = decode_workspace_size(B, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(workspace, "workspace")
    rc = lib().attn_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), _ptr(nk), B, Hq, Hkv, cap, d,
                           int(num_splits), _scale(scale, d), _ptr(lse_t), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "attn_decode")
    return out, lse_t


def attn_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                      nk: torch.Tensor, num_splits: int, scale: float | None = None,
                      workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      lse: torch.Tensor | bool | None = True, stream=None):
    """Paged decode. q [B, Hq, d]; pages [num_pages, page_size, Hkv, d]; block_table [B, max_pages]
    int32 and nk [B] int32 on the device."""
    if q.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [B, Hq, d], pages [num_pages, page_size, Hkv, d], block_table [B, max_pages]")
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape) or block_table.shape[0] != B:
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, d]; block_table [B, max_pages]")
    for t, n in ((q, "q"), (k_pages, "k_pages"), (v_pages, "v_pages")):
        _cuda(t, n, torch.bfloat16)
    _cuda(block_table, "block_table", torch.int32)
    _cuda(nk, "nk", torch.int32)
    if out is None:
        out = torch.empty_like(q)
    _cuda(out, "out", torch.bfloat16)
    lse_t = None
    if lse is True:
        lse_t = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    elif isinstance(lse, torch.Tensor):
        lse_t = lse
        _cuda(lse_t, "lse", torch.float32)
    need = decode_workspace_size(B, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(workspace, "workspace")
    rc = lib().attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(out), _ptr(block_table), _ptr(nk), B, Hq,
                                 Hkv, page_size, num_pages, block_table.shape[1], d, int(num_splits), _scale(scale, d),
                                 _ptr(lse_t), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(rc, "attn_decode_paged")
    return out, lse_t


_FP8_CODES = (torch.uint8, torch.float8_e4m3fn)


def _fp8_cache(k, v, k_scale, v_scale, Hkv, d, names):
    for t, n in ((k, names[0]), (v, names[1])):
        _cuda(t, n)
        if t.dtype not in _FP8_CODES:
            raise ValueError(f"{n} must hold E4M3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _cuda(t, n, torch.float32)
        if tuple(t.shape) != (Hkv, d):
            raise ValueError(f"{n} must be [Hkv, d] = [{Hkv}, {d}]")


def _decode_outputs(q, B, Hq, d, num_splits, out, lse, workspace):
    if out is None:
        out = torch.empty_like(q)
    _cuda(out, "out", torch.bfloat16)
    lse_t = None
    if lse is True:
        lse_t = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    elif isinstance(lse, torch.Tensor):
        lse_t = lse
        _cuda(lse_t, "lse", torch.float32)
    need = decode_workspace_size(B, Hq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(workspace, "workspace")
    return out, lse_t, workspace


def attn_decode_fp8(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, k_scale: torch.Tensor,
                    v_scale: torch.Tensor, nk: torch.Tensor, num_splits: int, scale: float | None = None,
                    workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | bool | None = True, stream=None):
    """Decode against an FP8 cache. q [B, Hq, d] bf16; caches [B, Hkv, cap, d] of E4M3 codes;
    k_scale, v_scale [Hkv, d] fp32 (value = e4m3(code) * scale[head, channel]); nk [B] int32."""
    if q.dim() != 3 or kcache.dim() != 4:
        raise ValueError("q must be [B, Hq, d] and caches [B, Hkv, cap, d]")
    B, Hq, d = q.shape
    Bk, Hkv, cap, dk = kcache.shape
    if Bk != B or dk != d or tuple(vcache.shape) != tuple(kcache.shape):
        raise ValueError("kcache and vcache must be [B, Hkv, cap, d] with q's B and d")
    _cuda(q, "q", torch.bfloat16)
    _fp8_cache(kcache, vcache, k_scale, v_scale, Hkv, d, ("kcache", "vcache"))
    _cuda(nk, "nk", torch.int32)
    out, lse_t, workspace = _decode_outputs(q, B, Hq, d, num_splits, out, lse, workspace)
    rc = lib().attn_decode_fp8(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(nk),
                               B, Hq, Hkv, cap, d, int(num_splits), _scale(scale, d), _ptr(lse_t), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "attn_decode_fp8")
    return out, lse_t


def attn_decode_paged_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                          v_scale: torch.Tensor, block_table: torch.Tensor, nk: torch.Tensor, num_splits: int,
                          scale: float | None = None, workspace: torch.Tensor | None = None,
                          out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = True, stream=None):
    """Paged decode against FP8 pages [num_pages, page_size, Hkv, d] of E4M3 codes."""
    if q.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [B, Hq, d], pages [num_pages, page_size, Hkv, d], block_table [B, max_pages]")
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = k_pages.shape
    if dk != d or tuple(v_pages.shape) != tuple(k_pages.shape) or block_table.shape[0] != B:
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, d]; block_table [B, max_pages]")
    _cuda(q, "q", torch.bfloat16)
    _fp8_cache(k_pages, v_pages, k_scale, v_scale, Hkv, d, ("k_pages", "v_pages"))
    _cuda(block_table, "block_table", torch.int32)
    _cuda(nk, "nk", torch.int32)
    out, lse_t, workspace = _decode_outputs(q, B, Hq, d, num_splits, out, lse, workspace)
    rc = lib().attn_decode_paged_fp8(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(out),
                                     _ptr(block_table), _ptr(nk), B, Hq, Hkv, page_size, num_pages,
                                     block_table.shape[1], d, int(num_splits), _scale(scale, d), _ptr(lse_t),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "attn_decode_paged_fp8")
    return out, lse_t


def varlen_workspace_size(num_seqs: int, max_seqlen_k: int, Hq: int, Hkv: int, d: int) -> int:
    return int(lib().attn_varlen_workspace_size(num_seqs, max_seqlen_k, Hq, Hkv, d))


def attn_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int, causal: bool = True,
                scale: float | None = None, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                lse: torch.Tensor | bool | None = True, stream=None, window: int = 0):
    """Packed varlen. q [total_q, Hq, d]; k, v [total_k, Hkv, d]; cu_seqlens int32 [num_seqs + 1] (device).

    ``window`` > 0 (causal only): sliding window of that many keys ending at each query's limit."""
    if window and not causal:
        raise ValueError("a sliding window needs causal=True")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [total_q, Hq, d] and k, v [total_k, Hkv, d]")
    tq, Hq, d = q.shape
    tk, Hkv, dk = k.shape
    if dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [total_k, Hkv, d] with q's d")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _cuda(t, n, torch.bfloat16)
    _cuda(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    _cuda(cu_seqlens_k, "cu_seqlens_k", torch.int32)
    num_seqs = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != num_seqs + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if out is None:
        out = torch.empty_like(q)
    _cuda(out, "out", torch.bfloat16)
    lse_t = None
    if lse is True:
        lse_t = torch.empty((tq, Hq), dtype=torch.float32, device=q.device)
    elif isinstance(lse, torch.Tensor):
        lse_t = lse
        _cuda(lse_t, "lse", torch.float32)
    need = varlen_workspace_size(num_seqs, int(max_seqlen_k), Hq, Hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(workspace, "workspace")
    if window:
        fn, mode, what = lib().attn_varlen_window, int(window), "attn_varlen_window"
    else:
        fn, mode, what = lib().attn_varlen, int(bool(causal)), "attn_varlen"
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse_t), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), num_seqs, tq,
            tk, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, d, mode, _scale(scale, d), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, what)
    return out, lse_t


# ---------------------------------------------------------------- speculative decoding


class _Call:
    """Where a call runs: the device of its tensors and ``stream`` (default: that device's current
    stream). What the call allocates belongs to that stream, so that its memory is not handed to
    other work while the kernels still run."""

    def __init__(self, device, stream):
        self.device = device
        self.here = device.index is None or device.index == torch.cuda.current_device()
        self.stream = torch.cuda.current_stream(device) if stream is None else stream
        self.guard = stream is not None or not self.here

    def __enter__(self):
        if self.guard:
            self.context = torch.cuda.stream(self.stream) if self.stream.device == self.device else None
            if self.context is None:
                raise ValueError(f"the stream is on {self.stream.device}, the tensors on {self.device}")
            self.context.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.guard:
            self.context.__exit__(*exc)


def _int32(t, name, device, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on {device}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t


def _out(t, name, device, dtype, shape):
    """An output tensor: a new one, or the caller's."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.dtype != dtype or t.device != device or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")
    return t


def _rows(t, name, device, heads, d):
    """bf16 [rows, heads, d] whose rows may lie apart (a slice of a fused projection): the row stride."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device != device or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D bf16 tensor on {device}")
    n, h, c = t.shape
    if (h, c) != (heads, d):
        raise ValueError(f"{name} must be [rows, {heads}, {d}], got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if n and ((s2 != 1 and c > 1) or (s1 != c and h > 1) or (n > 1 and (s0 < h * c or s0 % 8))):
        raise ValueError(f"{name}: heads must be contiguous, and rows a multiple of 8 elements apart")
    return s0 if n > 1 else h * c


def tree_workspace_size(num_seqs: int, max_nodes: int, Hq: int, Hkv: int, d: int) -> int:
    return int(lib().attn_tree_workspace_size(num_seqs, max_nodes, Hq, Hkv, d))


def _tree(q, k, v, table, k_new, v_new, nk, cu, mask, max_nodes, scale, workspace, out, lse, stream):
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise ValueError("q must be a CUDA tensor [total_q, Hq, d]")
    if k.dim() != 4 or tuple(v.shape) != tuple(k.shape) or k_new.dim() != 3:
        raise ValueError("the caches must be 4-D and alike; k_new and v_new [total_q, Hkv, d]")
    device = q.device
    tq, Hq, d = q.shape
    Hkv = k_new.shape[1]
    if table is None:
        num_seqs, hk, cap, dk = k.shape
    else:
        num_pages, page_size, hk, dk = k.shape
        num_seqs = table.shape[0]
        _int32(table, "block_table", device)
        if table.dim() != 2:
            raise ValueError("block_table must be [num_seqs, max_pages]")
    if dk != d or hk != Hkv:
        raise ValueError("q, the caches, k_new and v_new must agree in head dim and KV heads")
    for t, n in ((k, "k cache"), (v, "v cache")):
        _cuda(t, n, torch.bfloat16)
        if t.device != device:
            raise ValueError(f"the {n} must be on {device}")
    qs = _rows(q, "q", device, Hq, d)
    ks = _rows(k_new, "k_new", device, Hkv, d)
    vs = _rows(v_new, "v_new", device, Hkv, d)
    if k_new.shape[0] != tq or v_new.shape[0] != tq:
        raise ValueError("q, k_new and v_new must have the same number of rows")
    _int32(nk, "nk", device, (num_seqs,))
    _int32(cu, "cu_seqlens_q", device, (num_seqs + 1,))
    max_nodes = int(max_nodes)
    if mask.dtype not in (torch.int64, torch.uint64) or mask.device != device or not mask.is_contiguous() or \
            tuple(mask.shape) != (tq, (max_nodes + 63) // 64):
        raise ValueError("mask must be a contiguous int64 tensor [total_q, ceil(max_nodes / 64)]")
    with _Call(device, stream) as st:
        out = _out(out, "out", device, torch.bfloat16, (tq, Hq, d))
        lse_t = None
        if lse is True:
            lse_t = torch.empty((tq, Hq), dtype=torch.float32, device=device)
        elif isinstance(lse, torch.Tensor):
            lse_t = _out(lse, "lse", device, torch.float32, (tq, Hq))
        if workspace is None:
            workspace = torch.empty(max(tree_workspace_size(num_seqs, max_nodes, Hq, Hkv, d), 16), dtype=torch.uint8,
                                    device=device)
        _cuda(workspace, "workspace")
        if workspace.device != device:
            raise ValueError(f"workspace must be on {device}")
        ws_bytes = workspace.numel() * workspace.element_size()
        if table is None:
            rc = lib().attn_tree(_ptr(q), _ptr(k), _ptr(v), _ptr(k_new), _ptr(v_new), _ptr(out), _ptr(lse_t), _ptr(nk),
                                 _ptr(cu), _ptr(mask), num_seqs, tq, max_nodes, cap, Hq, Hkv, d, qs, ks, vs,
                                 _scale(scale, d), _ptr(workspace), ws_bytes, st)
        else:
            rc = lib().attn_tree_paged(_ptr(q), _ptr(k), _ptr(v), _ptr(table), _ptr(k_new), _ptr(v_new), _ptr(out),
                                       _ptr(lse_t), _ptr(nk), _ptr(cu), _ptr(mask), num_seqs, tq, max_nodes, page_size,
                                       num_pages, table.shape[1], Hq, Hkv, d, qs, ks, vs, _scale(scale, d),
                                       _ptr(workspace), ws_bytes, st)
        _check(rc, "attn_tree" if table is None else "attn_tree_paged")
    return out, lse_t


def attn_tree(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
              nk: torch.Tensor, cu_seqlens_q: torch.Tensor, mask: torch.Tensor, max_nodes: int,
              scale: float | None = None, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
              lse: torch.Tensor | bool | None = True, stream=None):
    """Drafted token trees over a contiguous cache. q [total_q, Hq, d], k_new, v_new [total_q, Hkv, d] bf16
    (rows may lie apart); caches [B, Hkv, cap, d]; nk [B], cu_seqlens_q [B + 1] int32; mask
    [total_q, ceil(max_nodes / 64)] int64 (``attn_tree_mask`` makes it) -> (o, lse or None)."""
    return _tree(q, kcache, vcache, None, k_new, v_new, nk, cu_seqlens_q, mask, max_nodes, scale, workspace, out, lse,
                 stream)


def attn_tree_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                    k_new: torch.Tensor, v_new: torch.Tensor, nk: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    mask: torch.Tensor, max_nodes: int, scale: float | None = None,
                    workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | bool | None = True, stream=None):
    """``attn_tree`` over a paged cache: pages [num_pages, page_size, Hkv, d], block_table [B, max_pages] int32."""
    return _tree(q, k_pages, v_pages, block_table, k_new, v_new, nk, cu_seqlens_q, mask, max_nodes, scale, workspace,
                 out, lse, stream)


def attn_tree_mask(parents: torch.Tensor, cu_seqlens_q: torch.Tensor, max_nodes: int, nk: torch.Tensor | None = None,
                   mask: torch.Tensor | None = None, positions: torch.Tensor | None = None, stream=None):
    """Masks and positions of drafted trees. parents [total_q] int32 (index within the sequence, a root
    outside [0, i)) -> (mask [total_q, ceil(max_nodes / 64)] int64, positions [total_q] int32 = nk + depth)."""
    if not isinstance(parents, torch.Tensor) or not parents.is_cuda or parents.dim() != 1:
        raise ValueError("parents must be a 1-D CUDA tensor")
    device, tq, max_nodes = parents.device, parents.shape[0], int(max_nodes)
    _int32(parents, "parents", device)
    _int32(cu_seqlens_q, "cu_seqlens_q", device)
    num_seqs = cu_seqlens_q.numel() - 1
    if nk is not None:
        _int32(nk, "nk", device, (num_seqs,))
    with _Call(device, stream) as st:
        mask = _out(mask, "mask", device, torch.int64, (tq, max(0, max_nodes + 63) // 64))
        positions = _out(positions, "positions", device, torch.int32, (tq,))
        rc = lib().attn_tree_mask(_ptr(parents), _ptr(cu_seqlens_q), _ptr(nk), _ptr(mask), _ptr(positions), num_seqs, tq,
                                  max_nodes, st)
        _check(rc, "attn_tree_mask")
    return mask, positions


def kv_plan_paged(nk: torch.Tensor, n_new: torch.Tensor, block_table: torch.Tensor, held: torch.Tensor,
                  free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, num_tokens: int, stream=None):
    """Room for n_new[b] further tokens of each request: extends block_table [B, max_pages] in place with
    pages from the top of the stack free_pages[:free_count] and returns (nk + n_new, held + pages taken,
    cu_seqlens [B + 1], slots [num_tokens], free_count - pages taken), all int32. A negative last value:
    the stack was short by so many pages, nothing of the plan may be used."""
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda or block_table.dim() != 2:
        raise ValueError("block_table must be a CUDA tensor [B, max_pages]")
    device, (B, max_pages) = block_table.device, block_table.shape
    _int32(block_table, "block_table", device)
    for t, n in ((nk, "nk"), (n_new, "n_new"), (held, "held")):
        _int32(t, n, device, (B,))
    _int32(free_pages, "free_pages", device)
    _int32(free_count, "free_count", device)
    if free_count.numel() != 1 or free_pages.dim() != 1:
        raise ValueError("free_pages must be 1-D and free_count one value")
    num_tokens = int(num_tokens)
    with _Call(device, stream) as st:
        if num_tokens < 0:
            raise ValueError("num_tokens must not be negative")
        nk_out, held_out = torch.empty_like(nk), torch.empty_like(held)
        cu = torch.empty(B + 1, dtype=torch.int32, device=device)
        slots = torch.empty(num_tokens, dtype=torch.int32, device=device)
        free_out = torch.empty_like(free_count)
        rc = lib().kv_plan_paged(_ptr(nk), _ptr(n_new), _ptr(block_table), _ptr(held), _ptr(free_pages), _ptr(free_count),
                                 _ptr(nk_out), _ptr(held_out), _ptr(cu), _ptr(slots), _ptr(free_out), B, int(page_size),
                                 max_pages, free_pages.numel(), num_tokens, st)
        _check(rc, "kv_plan_paged")
    return nk_out, held_out, cu, slots, free_out


def _append(k_new, v_new, slots, k_pages, v_pages, k_scale, v_scale, rows, stream, fp8):
    if not isinstance(k_pages, torch.Tensor) or not k_pages.is_cuda or k_pages.dim() != 4:
        raise ValueError("k_pages and v_pages must be CUDA tensors [num_pages, page_size, Hkv, d]")
    device = k_pages.device
    num_pages, page_size, Hkv, d = k_pages.shape
    if tuple(v_pages.shape) != tuple(k_pages.shape) or v_pages.device != device:
        raise ValueError("v_pages must be like k_pages")
    if fp8:
        _fp8_cache(k_pages, v_pages, k_scale, v_scale, Hkv, d, ("k_pages", "v_pages"))
        if k_scale.device != device or v_scale.device != device:
            raise ValueError(f"k_scale and v_scale must be on {device}")
    else:
        _cuda(k_pages, "k_pages", torch.bfloat16)
        _cuda(v_pages, "v_pages", torch.bfloat16)
    ks = _rows(k_new, "k_new", device, Hkv, d)
    vs = _rows(v_new, "v_new", device, Hkv, d)
    if v_new.shape[0] != k_new.shape[0]:
        raise ValueError("k_new and v_new must have the same number of rows")
    _int32(slots, "slots", device)
    n = slots.numel()
    if rows is not None:
        _int32(rows, "rows", device, tuple(slots.shape))
    with _Call(device, stream) as st:
        if fp8:
            rc = lib().kv_append_paged_fp8(_ptr(k_new), _ptr(v_new), _ptr(slots), _ptr(rows), _ptr(k_pages), _ptr(v_pages),
                                           _ptr(k_scale), _ptr(v_scale), n, k_new.shape[0], page_size, num_pages, Hkv, d,
                                           ks, vs, st)
        else:
            rc = lib().kv_append_paged(_ptr(k_new), _ptr(v_new), _ptr(slots), _ptr(rows), _ptr(k_pages), _ptr(v_pages), n,
                                       k_new.shape[0], page_size, num_pages, Hkv, d, ks, vs, st)
        _check(rc, "kv_append_paged_fp8" if fp8 else "kv_append_paged")
    return k_pages, v_pages


def kv_append_paged(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor,
                    v_pages: torch.Tensor, rows: torch.Tensor | None = None, stream=None):
    """Writes K and V rows [n, Hkv, d] bf16 into the pages: slot slots[i] takes row rows[i] (default i);
    slots and rows out of range are skipped. Returns (k_pages, v_pages), written in place."""
    return _append(k_new, v_new, slots, k_pages, v_pages, None, None, rows, stream, False)


def kv_append_paged_fp8(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor,
                        v_pages: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                        rows: torch.Tensor | None = None, stream=None):
    """``kv_append_paged`` into pages of E4M3 codes: code = nearest E4M3 value of x / scale[head, channel]."""
    return _append(k_new, v_new, slots, k_pages, v_pages, k_scale, v_scale, rows, stream, True)


def get_status(stream=None) -> int:
    """Synchronises the stream; BWATTN_ERR_TIMEOUT if a kernel gave up a wait, else OK."""
    return int(lib().bwattn_get_status(_stream(stream)))


def clear_status(stream=None) -> None:
    _check(lib().bwattn_clear_status(_stream(stream)), "bwattn_clear_status")


def set_wait_timeout_ns(ns: int) -> None:
    lib().bwattn_set_wait_timeout_ns(int(ns))


def test_wait_timeout(stream=None) -> None:
    _check(lib().bwattn_test_wait_timeout(_stream(stream)), "bwattn_test_wait_timeout")


def launch_count() -> int:
    return int(lib().bwattn_launch_count())
