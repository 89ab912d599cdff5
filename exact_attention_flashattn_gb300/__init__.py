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
* Around a paged cache's attention: ``attn_qk_norm_rope`` (per-head norm and rotation of q and k),
  ``attn_chunk_paged`` (new tokens over the pages), ``attn_tree_verify`` (which drafts are kept).
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
    "tree_workspace_size", "attn_chunk_paged", "chunk_workspace_size", "attn_qk_norm_rope", "attn_tree_verify",
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
        L.attn_chunk_workspace_size.argtypes = [ci] * 5
        L.attn_chunk_workspace_size.restype = sz
        L.attn_chunk_paged.argtypes = [vp] * 8 + [ci] * 9 + [i64, ci, cf, vp, sz, vp]
        L.attn_chunk_paged.restype = ci
        L.attn_qk_norm_rope.argtypes = [vp] * 9 + [cf] + [ci] * 7 + [i64] * 4 + [vp]
        L.attn_qk_norm_rope.restype = ci
        L.attn_tree_verify.argtypes = [vp] * 10 + [ci] * 4 + [i64] * 2 + [vp]
        L.attn_tree_verify.restype = ci
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


# These calls run at every step of a server, where the host's time counts: devices are compared by
# index, the current stream is read as its raw handle (a Stream object costs 2 us), and nothing is
# entered when the tensors' device is current and no stream is named.

_I32, _BF16, _F32, _Tensor = torch.int32, torch.bfloat16, torch.float32, torch.Tensor
# the current device, and its current stream's handle (a Stream object takes 2 us; absent in a CPU-only torch)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(fn, dev: int, stream, *args):
    """``fn`` with the handle of the call's stream: the current one of device ``dev``, or ``stream``. What a
    call allocates belongs to its stream, so that the memory is not handed to other work while the kernels
    still run."""
    if stream is None:
        if dev == _current_device():
            return fn(_raw_stream(dev), dev, *args)
        stream = torch.cuda.current_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    with torch.cuda.stream(stream):
        return fn(stream.cuda_stream, dev, *args)


def _first(t, name, ndim):
    """The device index of a call's leading tensor."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dim() != ndim:
        raise ValueError(f"{name} must be a {ndim}-D CUDA tensor")
    return t.get_device()


def _like(t, name, dev, dtype, shape=None):
    """A contiguous tensor of that type on the call's device: its address."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _out(t, name, dev, dtype, shape):
    """An output tensor: a new one, or the caller's."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _like(t, name, dev, dtype, shape)
    return t


def _rows(t, name, dev, shape):
    """bf16 [rows, heads, d] whose rows may lie apart (a slice of a fused projection): the row stride."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be a bf16 tensor {shape} on cuda:{dev}")
    n, h, c = shape
    if t.is_contiguous():
        return h * c
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != c and h > 1) or (n > 1 and (s0 < h * c or s0 % 8)):
        raise ValueError(f"{name}: heads must be contiguous, and rows a multiple of 8 elements apart")
    return s0 if n > 1 else h * c


def tree_workspace_size(num_seqs: int, max_nodes: int, Hq: int, Hkv: int, d: int) -> int:
    return int(lib().attn_tree_workspace_size(num_seqs, max_nodes, Hq, Hkv, d))


def _tree(st, dev, q, k, v, table, k_new, v_new, nk, cu, mask, max_nodes, scale, workspace, out, lse):
    tq, Hq, d = q.shape
    if table is None:
        num_seqs, Hkv, cap, dk = k.shape
    else:
        num_pages, page_size, Hkv, dk = k.shape
        num_seqs, max_pages = table.shape
        tp = _like(table, "block_table", dev, _I32)
    if dk != d:
        raise ValueError("q and the caches must have the same head dim")
    kp = _like(k, "the k cache", dev, _BF16)
    vp = _like(v, "the v cache", dev, _BF16, k.shape)
    qs = _rows(q, "q", dev, q.shape)
    ks = _rows(k_new, "k_new", dev, (tq, Hkv, d))
    vs = _rows(v_new, "v_new", dev, (tq, Hkv, d))
    nkp = _like(nk, "nk", dev, _I32, (num_seqs,))
    cup = _like(cu, "cu_seqlens_q", dev, _I32, (num_seqs + 1,))
    if isinstance(mask, torch.Tensor) and mask.dtype is torch.uint64:
        mask = mask.view(torch.int64)
    mp = _like(mask, "mask", dev, torch.int64, (tq, (max_nodes + 63) // 64))
    out = _out(out, "out", dev, _BF16, q.shape)
    if lse is True:
        lse = torch.empty((tq, Hq), dtype=_F32, device=dev)
    elif not isinstance(lse, torch.Tensor):
        lse = None
    else:
        _like(lse, "lse", dev, _F32, (tq, Hq))
    if workspace is None:
        workspace = torch.empty(max(tree_workspace_size(num_seqs, max_nodes, Hq, Hkv, d), 16), dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    scale = _scale(scale, d)
    lp = None if lse is None else lse.data_ptr()
    wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    L = _lib or lib()
    if table is None:
        rc = L.attn_tree(q.data_ptr(), kp, vp, k_new.data_ptr(), v_new.data_ptr(), out.data_ptr(), lp, nkp, cup, mp,
                         num_seqs, tq, max_nodes, cap, Hq, Hkv, d, qs, ks, vs, scale, wp, wb, st)
    else:
        rc = L.attn_tree_paged(q.data_ptr(), kp, vp, tp, k_new.data_ptr(), v_new.data_ptr(), out.data_ptr(), lp, nkp, cup,
                               mp, num_seqs, tq, max_nodes, page_size, num_pages, max_pages, Hq, Hkv, d, qs, ks, vs, scale,
                               wp, wb, st)
    if rc:
        _check(rc, "attn_tree" if table is None else "attn_tree_paged")
    return out, lse


def attn_tree(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
              nk: torch.Tensor, cu_seqlens_q: torch.Tensor, mask: torch.Tensor, max_nodes: int,
              scale: float | None = None, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
              lse: torch.Tensor | bool | None = True, stream=None):
    """Drafted token trees over a contiguous cache. q [total_q, Hq, d], k_new, v_new [total_q, Hkv, d] bf16
    (rows may lie apart); caches [B, Hkv, cap, d]; nk [B], cu_seqlens_q [B + 1] int32; mask
    [total_q, ceil(max_nodes / 64)] int64 (``attn_tree_mask`` makes it) -> (o, lse or None)."""
    dev = _first(q, "q", 3)
    _first(kcache, "kcache", 4)
    return _run(_tree, dev, stream, q, kcache, vcache, None, k_new, v_new, nk, cu_seqlens_q, mask, int(max_nodes),
                scale, workspace, out, lse)


def attn_tree_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                    k_new: torch.Tensor, v_new: torch.Tensor, nk: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    mask: torch.Tensor, max_nodes: int, scale: float | None = None,
                    workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | bool | None = True, stream=None):
    """``attn_tree`` over a paged cache: pages [num_pages, page_size, Hkv, d], block_table [B, max_pages] int32."""
    dev = _first(q, "q", 3)
    _first(k_pages, "k_pages", 4)
    _first(block_table, "block_table", 2)
    return _run(_tree, dev, stream, q, k_pages, v_pages, block_table, k_new, v_new, nk, cu_seqlens_q, mask,
                int(max_nodes), scale, workspace, out, lse)


def attn_tree_mask(parents: torch.Tensor, cu_seqlens_q: torch.Tensor, max_nodes: int, nk: torch.Tensor | None = None,
                   mask: torch.Tensor | None = None, positions: torch.Tensor | None = None, stream=None):
    """Masks and positions of drafted trees. parents [total_q] int32 (index within the sequence, a root
    outside [0, i)) -> (mask [total_q, ceil(max_nodes / 64)] int64, positions [total_q] int32 = nk + depth)."""
    dev = _first(parents, "parents", 1)
    return _run(_tree_mask, dev, stream, parents, cu_seqlens_q, int(max_nodes), nk, mask, positions)


def _tree_mask(st, dev, parents, cu, max_nodes, nk, mask, positions):
    tq, num_seqs = parents.shape[0], cu.numel() - 1
    pp = _like(parents, "parents", dev, _I32)
    cup = _like(cu, "cu_seqlens_q", dev, _I32)
    nkp = None if nk is None else _like(nk, "nk", dev, _I32, (num_seqs,))
    mask = _out(mask, "mask", dev, torch.int64, (tq, max(0, max_nodes + 63) // 64))
    positions = _out(positions, "positions", dev, _I32, (tq,))
    rc = (_lib or lib()).attn_tree_mask(pp, cup, nkp, mask.data_ptr(), positions.data_ptr(), num_seqs, tq, max_nodes, st)
    if rc:
        _check(rc, "attn_tree_mask")
    return mask, positions


def kv_plan_paged(nk: torch.Tensor, n_new: torch.Tensor, block_table: torch.Tensor, held: torch.Tensor,
                  free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, num_tokens: int, stream=None):
    """Room for n_new[b] further tokens of each request: extends block_table [B, max_pages] in place with
    pages from the top of the stack free_pages[:free_count] and returns (nk + n_new, held + pages taken,
    cu_seqlens [B + 1], slots [num_tokens], free_count - pages taken), all int32. A negative last value:
    the stack was short by so many pages, nothing of the plan may be used."""
    dev = _first(block_table, "block_table", 2)
    return _run(_plan, dev, stream, nk, n_new, block_table, held, free_pages, free_count, int(page_size), int(num_tokens))


def _plan(st, dev, nk, n_new, table, held, free_pages, free_count, page_size, num_tokens):
    B, max_pages = table.shape
    if num_tokens < 0 or free_pages.dim() != 1:
        raise ValueError("num_tokens must not be negative, free_pages 1-D")
    args = (_like(nk, "nk", dev, _I32, (B,)), _like(n_new, "n_new", dev, _I32, (B,)), _like(table, "block_table", dev, _I32),
            _like(held, "held", dev, _I32, (B,)), _like(free_pages, "free_pages", dev, _I32),
            _like(free_count, "free_count", dev, _I32))
    if free_count.numel() != 1:
        raise ValueError("free_count must be one value")
    nk_out, held_out, free_out, cu, slots = [torch.empty(n, dtype=_I32, device=dev)
                                             for n in (B, B, free_count.shape, B + 1, num_tokens)]
    rc = (_lib or lib()).kv_plan_paged(*args, nk_out.data_ptr(), held_out.data_ptr(), cu.data_ptr(), slots.data_ptr(),
                                       free_out.data_ptr(), B, page_size, max_pages, free_pages.numel(), num_tokens, st)
    if rc:
        _check(rc, "kv_plan_paged")
    return nk_out, held_out, cu, slots, free_out


def _append(st, dev, k_new, v_new, slots, k_pages, v_pages, k_scale, v_scale, rows, fp8):
    num_pages, page_size, Hkv, d = k_pages.shape
    dtype = k_pages.dtype
    if dtype not in _FP8_CODES if fp8 else dtype is not _BF16:
        raise ValueError("pages must hold " + ("E4M3 codes (uint8 or float8_e4m3fn)" if fp8 else "bf16") + f", got {dtype}")
    kp = _like(k_pages, "k_pages", dev, dtype)
    vp = _like(v_pages, "v_pages", dev, dtype, k_pages.shape)
    n = k_new.shape[0]
    ks = _rows(k_new, "k_new", dev, (n, Hkv, d))
    vs = _rows(v_new, "v_new", dev, (n, Hkv, d))
    sp = _like(slots, "slots", dev, _I32)
    rp = None if rows is None else _like(rows, "rows", dev, _I32, slots.shape)
    L = _lib or lib()
    if fp8:
        scales = (_like(k_scale, "k_scale", dev, _F32, (Hkv, d)), _like(v_scale, "v_scale", dev, _F32, (Hkv, d)))
        rc = L.kv_append_paged_fp8(k_new.data_ptr(), v_new.data_ptr(), sp, rp, kp, vp, *scales, slots.numel(), n, page_size,
                                   num_pages, Hkv, d, ks, vs, st)
    else:
        rc = L.kv_append_paged(k_new.data_ptr(), v_new.data_ptr(), sp, rp, kp, vp, slots.numel(), n, page_size, num_pages,
                               Hkv, d, ks, vs, st)
    if rc:
        _check(rc, "kv_append_paged_fp8" if fp8 else "kv_append_paged")
    return k_pages, v_pages


def kv_append_paged(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor,
                    v_pages: torch.Tensor, rows: torch.Tensor | None = None, stream=None):
    """Writes K and V rows [n, Hkv, d] bf16 into the pages: slot slots[i] takes row rows[i] (default i);
    slots and rows out of range are skipped. Returns (k_pages, v_pages), written in place."""
    dev = _first(k_pages, "k_pages", 4)
    _first(k_new, "k_new", 3)
    return _run(_append, dev, stream, k_new, v_new, slots, k_pages, v_pages, None, None, rows, False)


def kv_append_paged_fp8(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor,
                        v_pages: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                        rows: torch.Tensor | None = None, stream=None):
    """``kv_append_paged`` into pages of E4M3 codes: code = nearest E4M3 value of x / scale[head, channel]."""
    dev = _first(k_pages, "k_pages", 4)
    _first(k_new, "k_new", 3)
    return _run(_append, dev, stream, k_new, v_new, slots, k_pages, v_pages, k_scale, v_scale, rows, True)


# ---------------------------------------------------------------- around a paged cache's attention


def chunk_workspace_size(num_seqs: int, max_seqlen_q: int, Hq: int, Hkv: int, d: int) -> int:
    return int(lib().attn_chunk_workspace_size(num_seqs, max_seqlen_q, Hq, Hkv, d))


def attn_chunk_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                     nk: torch.Tensor, cu_seqlens_q: torch.Tensor, max_seqlen_q: int, causal: bool = True,
                     scale: float | None = None, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | bool | None = True, stream=None):
    """New tokens over a paged cache that holds their own keys too. q [total_q, Hq, d] bf16 (rows may lie apart);
    pages [num_pages, page_size, Hkv, d], block_table [B, max_pages] int32; nk [B] (keys, the new tokens' among
    them), cu_seqlens_q [B + 1] int32 -> (o, lse or None). ``causal`` False: every token sees all nk keys."""
    dev = _first(q, "q", 3)
    _first(k_pages, "k_pages", 4)
    _first(block_table, "block_table", 2)
    return _run(_chunk, dev, stream, q, k_pages, v_pages, block_table, nk, cu_seqlens_q, int(max_seqlen_q), bool(causal),
                scale, workspace, out, lse)


def _chunk(st, dev, q, k, v, table, nk, cu, most, causal, scale, workspace, out, lse):
    tq, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = k.shape
    num_seqs, max_pages = table.shape
    if dk != d:
        raise ValueError("q and the pages must have the same head dim")
    tp = _like(table, "block_table", dev, _I32)
    kp = _like(k, "k_pages", dev, _BF16)
    vp = _like(v, "v_pages", dev, _BF16, k.shape)
    qs = _rows(q, "q", dev, q.shape)
    nkp = _like(nk, "nk", dev, _I32, (num_seqs,))
    cup = _like(cu, "cu_seqlens_q", dev, _I32, (num_seqs + 1,))
    out = torch.empty_like(q) if out is None else _out(out, "out", dev, _BF16, q.shape)
    if lse is True:
        lse = torch.empty((tq, Hq), dtype=_F32, device=dev)
    elif not isinstance(lse, _Tensor):
        lse = None
    else:
        _like(lse, "lse", dev, _F32, (tq, Hq))
    if workspace is None:
        workspace = torch.empty(max(chunk_workspace_size(num_seqs, most, Hq, Hkv, d), 16), dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    rc = (_lib or lib()).attn_chunk_paged(
        q.data_ptr(), kp, vp, tp, out.data_ptr(), None if lse is None else lse.data_ptr(), nkp, cup, num_seqs, tq, most,
        page_size, num_pages, max_pages, Hq, Hkv, d, qs, causal, _scale(scale, d), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), st)
    if rc:
        _check(rc, "attn_chunk_paged")
    return out, lse


def attn_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor,
                      q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                      axes: torch.Tensor | None = None, interleaved: bool = False, q_out: torch.Tensor | None = None,
                      k_out: torch.Tensor | None = None, stream=None):
    """Per-head norm and rotation of q [n, Hq, d] and k [n, Hkv, d] bf16 (rows may lie apart) -> (q_out, k_out), which may
    be q and k themselves. positions [n] or [num_axes, n] int32; inv_freq [pairs] fp32; axes [pairs] int32, each
    pair's row of positions; weights [d] bf16 (None: no norm). Pairs are channels (i, i + pairs), or neighbours
    with ``interleaved``; channels behind them are not rotated."""
    dev = _first(q, "q", 3)
    _first(k, "k", 3)
    return _run(_qk_rope, dev, stream, q, k, positions, inv_freq, q_weight, k_weight, float(eps), axes, bool(interleaved),
                q_out, k_out)


def _qk_rope(st, dev, q, k, positions, freq, q_weight, k_weight, eps, axes, interleaved, q_out, k_out):
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    qs, ks = _rows(q, "q", dev, q.shape), _rows(k, "k", dev, (n, Hkv, d))
    num_axes = 1 if positions.dim() == 1 else positions.shape[0]
    pp = _like(positions, "positions", dev, _I32, (n,) if positions.dim() == 1 else (num_axes, n))
    if freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D")
    fp = _like(freq, "inv_freq", dev, _F32)
    pairs = freq.shape[0]
    ap = None if axes is None else _like(axes, "axes", dev, _I32, (pairs,))
    qw = None if q_weight is None else _like(q_weight, "q_weight", dev, _BF16, (d,))
    kw = None if k_weight is None else _like(k_weight, "k_weight", dev, _BF16, (d,))
    # (empty_like() of rows that lie apart is contiguous; two empty() take the host 1.5 us more)
    if q_out is None:
        q_out, qos = torch.empty_like(q), Hq * d
    else:
        qos = _rows(q_out, "q_out", dev, q.shape)
    if k_out is None:
        k_out, kos = torch.empty_like(k), Hkv * d
    else:
        kos = _rows(k_out, "k_out", dev, k.shape)
    rc = (_lib or lib()).attn_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), pp, ap, fp, qw, kw,
                                           eps, n, num_axes, pairs, interleaved, Hq, Hkv, d, qs, ks, qos, kos, st)
    if rc:
        _check(rc, "attn_qk_norm_rope")
    return q_out, k_out


def attn_tree_verify(tokens: torch.Tensor, parents: torch.Tensor, cu_seqlens_q: torch.Tensor, target_probs: torch.Tensor,
                     uniforms: torch.Tensor, sample_uniforms: torch.Tensor, max_nodes: int,
                     draft_probs: torch.Tensor | None = None, accepted: torch.Tensor | None = None,
                     counts: torch.Tensor | None = None, next_tokens: torch.Tensor | None = None, stream=None):
    """Which drafts are kept: tokens, parents [total_q] int32 (node 0 of a request its root), target_probs (and
    draft_probs, if the drafts were drawn from them) [total_q, vocab] fp32 (rows may lie apart), uniforms [total_q]
    and sample_uniforms [B] fp32 -> int32 (accepted [total_q]: packed rows of each request's path, then -1; counts
    [B]; next_tokens [B]), new or the caller's."""
    dev = _first(target_probs, "target_probs", 2)
    return _run(_verify, dev, stream, tokens, parents, cu_seqlens_q, target_probs, uniforms, sample_uniforms, int(max_nodes),
                draft_probs, accepted, counts, next_tokens)


def _prob_rows(t, name, dev, shape):
    """fp32 [rows, vocab] whose rows may lie apart: the row stride."""
    if not isinstance(t, _Tensor) or t.dtype is not _F32 or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name} must be an fp32 tensor {tuple(shape)} on cuda:{dev}")
    n, c = shape
    if t.is_contiguous() or n <= 1 and t.stride(1) == 1:
        return c
    if t.stride(1) != 1 or t.stride(0) < c:
        raise ValueError(f"{name}: a row's values must be contiguous, and rows must not overlap")
    return t.stride(0)


def _verify(st, dev, tokens, parents, cu, p, u, w, max_nodes, q, accepted, counts, following):
    n, vocab = p.shape
    num_seqs = cu.numel() - 1
    ps = _prob_rows(p, "target_probs", dev, p.shape)
    qs = 0 if q is None else _prob_rows(q, "draft_probs", dev, p.shape)
    args = (_like(tokens, "tokens", dev, _I32, (n,)), _like(parents, "parents", dev, _I32, (n,)),
            _like(cu, "cu_seqlens_q", dev, _I32), p.data_ptr(), None if q is None else q.data_ptr(),
            _like(u, "uniforms", dev, _F32, (n,)), _like(w, "sample_uniforms", dev, _F32, (num_seqs,)))
    # (after an empty() with a device's index a launch takes the host 1.5 us more than after an empty_like())
    accepted = torch.empty_like(tokens) if accepted is None else _out(accepted, "accepted", dev, _I32, (n,))
    counts = torch.empty_like(w, dtype=_I32) if counts is None else _out(counts, "counts", dev, _I32, (num_seqs,))
    following = torch.empty_like(w, dtype=_I32) if following is None else _out(following, "next_tokens", dev, _I32, (num_seqs,))
    rc = (_lib or lib()).attn_tree_verify(*args, accepted.data_ptr(), counts.data_ptr(), following.data_ptr(), num_seqs, n,
                                          max_nodes, vocab, ps, qs, st)
    if rc:
        _check(rc, "attn_tree_verify")
    return accepted, counts, following


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
