"""Python binding of the C ABI in include/fd.h (ctypes; marshalling only).

Every function takes CUDA torch tensors, checks that their dtype, shape,
contiguity and device fit the C call, passes raw device pointers and the
current CUDA stream, and turns a non-OK status into an exception.  All the
arithmetic runs in the CUDA kernels of ``libfd.so``; there is no fallback:
if the library is missing or no GPU is present, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

from . import _build_lib

FD_OK = 0
STATUS_NAMES = {0: "FD_OK", 1: "FD_ERR_INVALID_ARG", 2: "FD_ERR_UNSUPPORTED",
                3: "FD_ERR_WORKSPACE", 4: "FD_ERR_CUDA", 5: "FD_ERR_DEVICE_TIMEOUT",
                6: "FD_ERR_SCRATCH_TOO_SMALL", 7: "FD_ERR_BAD_PAGE", 8: "FD_ERR_BAD_OFFSETS",
                9: "FD_ERR_BAD_INDEX"}

INT_MAX = 2 ** 31 - 1

DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

# every symbol include/fd.h declares
EXPORTS = ["fd_status_str", "fd_version", "fd_num_sms", "fd_auto_num_splits",
           "fd_workspace_size", "fd_decode", "fd_decode_split", "fd_combine_mlo",
           "fd_combine_lse", "fd_device_status", "fd_decode_noalloc", "fd_decode_paged",
           "fd_decode_fp8", "fd_merge_lse", "fd_decode_gqa", "fd_workspace_size_gqa",
           "fd_selftest_wait_timeout", "fd_decode_gqa_paged", "fd_decode_gqa_fp8",
           "fd_decode_gqa_paged_fp8", "fd_resize_pages", "fd_append_paged", "fd_append_paged_fp8",
           "fd_append_rope_paged", "fd_append_rope_paged_fp8", "fd_workspace_size_extend", "fd_prefill", "fd_extend_paged", "fd_extend_paged_fp8",
           "fd_workspace_size_beam", "fd_beam_select", "fd_workspace_size_reorder", "fd_reorder_pages", "fd_copy_pages"]

_lock = threading.Lock()
_lib = None


class FDError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


def library_path() -> str:
    return _build_lib.LIB


def load(build_if_missing: bool = False):
    """Load libfd.so (no GPU needed).  Raises if it is not built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if build_if_missing and _build_lib.is_stale():
            _build_lib.build()
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library {path} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fd_status_str.argtypes = [I]
        lib.fd_status_str.restype = ctypes.c_char_p
        lib.fd_version.argtypes = []
        lib.fd_version.restype = I
        lib.fd_num_sms.argtypes = []
        lib.fd_num_sms.restype = I
        lib.fd_auto_num_splits.argtypes = [I, I, I, I, I, I]
        lib.fd_auto_num_splits.restype = I
        lib.fd_workspace_size.argtypes = [I, I, I, I, I]
        lib.fd_workspace_size.restype = S
        lib.fd_decode.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, I, P, P, S, P]
        lib.fd_decode.restype = I
        lib.fd_decode_split.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, P]
        lib.fd_decode_split.restype = I
        lib.fd_combine_mlo.argtypes = [P, P, P, I, I, I, I, P, I, P, P]
        lib.fd_combine_mlo.restype = I
        lib.fd_combine_lse.argtypes = [P, P, I, I, I, I, P, I, P, P]
        lib.fd_combine_lse.restype = I
        lib.fd_decode_paged.argtypes = [P, P, P, P, P, I, I, I, I, I, ctypes.c_longlong, I, I, F, P, I,
                                        P, P, S, P]
        lib.fd_decode_paged.restype = I
        lib.fd_decode_fp8.argtypes = [P, I, P, P, P, P, P, I, I, I, I, I, F, P, I, P, P, S, P]
        lib.fd_decode_fp8.restype = I
        lib.fd_merge_lse.argtypes = [P, P, P, P, I, I, P, P, P]
        lib.fd_merge_lse.restype = I
        lib.fd_decode_gqa.argtypes = [P, P, P, P, I, I, I, I, I, I, I, F, P, I, P, P, S, P]
        lib.fd_decode_gqa.restype = I
        lib.fd_workspace_size_gqa.argtypes = [I, I, I, I, I, I]
        lib.fd_workspace_size_gqa.restype = S
        lib.fd_device_status.argtypes = [I]
        lib.fd_device_status.restype = I
        lib.fd_selftest_wait_timeout.argtypes = [P]
        lib.fd_selftest_wait_timeout.restype = I
        lib.fd_decode_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, I, P, P]
        lib.fd_decode_noalloc.restype = I
        lib.fd_decode_gqa_paged.argtypes = [P, P, P, P, P, I, I, I, I, I, I, ctypes.c_longlong, I, I,
                                            F, P, I, P, P, S, P]
        lib.fd_decode_gqa_paged.restype = I
        lib.fd_decode_gqa_fp8.argtypes = [P, I, P, P, P, P, P, I, I, I, I, I, I, F, P, I, P, P, S, P]
        lib.fd_decode_gqa_fp8.restype = I
        lib.fd_decode_gqa_paged_fp8.argtypes = [P, I, P, P, P, P, P, P, I, I, I, I, I, I, ctypes.c_longlong, I,
                                                F, P, I, P, P, S, P]
        lib.fd_decode_gqa_paged_fp8.restype = I
        L = ctypes.c_longlong
        lib.fd_resize_pages.argtypes = [P, P, I, P, I, P, P, I, I, P, P, I, P, P]
        lib.fd_resize_pages.restype = I
        lib.fd_append_paged.argtypes = [P, P, P, I, I, I, L, L, I, P, P, I, L, P]
        lib.fd_append_paged.restype = I
        lib.fd_append_paged_fp8.argtypes = [P, P, P, P, P, P, I, I, I, I, L, L, I, P, P, I, L, P]
        lib.fd_append_paged_fp8.restype = I
        lib.fd_append_rope_paged.argtypes = [P] * 6 + [I] * 7 + [L, L, L, I, P, L, P, P, I, L, P]
        lib.fd_append_rope_paged.restype = I
        lib.fd_append_rope_paged_fp8.argtypes = [P] * 9 + [I] * 8 + [L, L, L, I, P, L, P, P, I, L, P]
        lib.fd_append_rope_paged_fp8.restype = I
        lib.fd_workspace_size_extend.argtypes = [I, I, I, I, I]
        lib.fd_workspace_size_extend.restype = S
        lib.fd_prefill.argtypes = [P, P, P, P, P, I, I, I, I, I, I, L, L, L, I, I, F, P, I, P, P, S, P]
        lib.fd_prefill.restype = I
        lib.fd_extend_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, I, L, I, I, L, I, F, P, I, P, P, S, P]
        lib.fd_extend_paged.restype = I
        lib.fd_extend_paged_fp8.argtypes = [P, I, P, P, P, P, P, P, P, I, I, I, I, I, L, I, I, L, F, P, I, P, P, S, P]
        lib.fd_extend_paged_fp8.restype = I
        lib.fd_workspace_size_beam.argtypes = [I, I, I, I]
        lib.fd_workspace_size_beam.restype = S
        lib.fd_beam_select.argtypes = [P, I, L, L, P, P, I, I, I, I, I, P, P, P, P, P, S, P]
        lib.fd_beam_select.restype = I
        lib.fd_workspace_size_reorder.argtypes = [I, I, I]
        lib.fd_workspace_size_reorder.restype = S
        lib.fd_reorder_pages.argtypes = [P, I, I, P, P, I, P, P, I, I, P, P, P, S, P]
        lib.fd_reorder_pages.restype = I
        lib.fd_copy_pages.argtypes = [P, I, I, I, I, P, P, I, L, P]
        lib.fd_copy_pages.restype = I
        _lib = lib
        return lib


def status_str(status: int) -> str:
    try:
        return load().fd_status_str(int(status)).decode()
    except Exception:  # pragma: no cover - library not loadable
        return STATUS_NAMES.get(status, str(status))


def _check(status: int, what: str) -> None:
    if status != FD_OK:
        raise FDError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (the library has no CPU path)")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _check_qkv(q, k, v, seqlens):
    _need_cuda(q, k, v, seqlens)
    if q.dtype not in DTYPE_CODE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, K, V must share one dtype among float32/float16/bfloat16")
    if k.dim() != 4 or v.shape != k.shape or q.shape != (k.shape[0], k.shape[1], k.shape[3]):
        raise ValueError(f"shapes: q{tuple(q.shape)} must be [B,H,d], K/V{tuple(k.shape)} [B,H,N,d]")
    if seqlens is not None and (seqlens.dtype != torch.int32 or seqlens.shape != (k.shape[0],)):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    B, H, N, d = k.shape
    return B, H, N, d


def num_sms() -> int:
    return load().fd_num_sms()


KV_DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, "f32": 0, "f16": 1,
                 "bf16": 2, "e4m3": 3}


def auto_num_splits(B, H, N, d, dtype=torch.bfloat16, sm_count=None) -> int:
    """fd_auto_num_splits: the split count of the two-call path for this
    shape and K/V storage type (a torch dtype, or "f32"/"f16"/"bf16"/"e4m3")."""
    sm = num_sms() if sm_count is None else sm_count
    return load().fd_auto_num_splits(B, H, N, d, KV_DTYPE_CODE[dtype], sm)


def workspace_size(B, H, N, d, num_splits=0) -> int:
    return load().fd_workspace_size(B, H, N, d, num_splits)


def new_workspace(B, H, N, d, num_splits=0, device=None) -> torch.Tensor:
    """A workspace for fd_decode (reusable across calls on one stream)."""
    n = workspace_size(B, H, N, d, num_splits)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


_ws_cache: dict = {}


def _cached_workspace(device, nbytes):
    key = (device.index if device.index is not None else torch.cuda.current_device())
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def decode(q, k, v, seqlens=None, num_splits=0, scale=None, out_dtype=None, out=None,
           lse=None, return_lse=True, workspace=None, stream=None):
    """Fused split-KV decode attention (fd_decode).  Returns ``(out, lse)``.

    q [B,H,d], k/v [B,H,N,d] on one CUDA device; ``seqlens`` int32 [B] or
    None; ``num_splits`` 0 = automatic.  ``workspace`` defaults to a cached
    buffer per device (calls that overlap on the GPU need their own
    workspaces).
    """
    B, H, N, d = _check_qkv(q, k, v, seqlens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, H, d), dtype=odt, device=q.device)
    _need_cuda(out, lse)
    if out.dtype not in DTYPE_CODE or out.shape != (B, H, d):
        raise ValueError("out must be [B,H,d] float32/float16/bfloat16")
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (B, H)):
        raise ValueError("lse must be float32 [B,H]")
    lib = load()
    need = lib.fd_workspace_size(B, H, N, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    _need_cuda(workspace)
    st = lib.fd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, H, N, d, DTYPE_CODE[q.dtype],
                       int(num_splits), float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(lse),
                       _ptr(workspace), workspace.numel() * workspace.element_size(),
                       _stream(q, stream))
    _check(st, "fd_decode")
    return out, lse



def decode_noalloc(q, k, v, seqlens=None, num_splits=0, scale=None, out_dtype=None, out=None,
                   lse=None, return_lse=True, stream=None):
    """fd_decode on the library's own device scratch (fd_decode_noalloc).
    Returns ``(out, lse)``.

    The C call allocates nothing.  This wrapper allocates only what the
    caller leaves out: pass ``out`` (and ``lse``, or ``return_lse=False``)
    for a call that allocates no device memory at all.  Calls on one device
    share the scratch, so they must not overlap on the GPU; problems whose
    partials exceed the scratch raise FD_ERR_SCRATCH_TOO_SMALL."""
    B, H, N, d = _check_qkv(q, k, v, seqlens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, H, d), dtype=odt, device=q.device)
    _need_cuda(out, lse)
    if out.dtype not in DTYPE_CODE or out.shape != (B, H, d):
        raise ValueError("out must be [B,H,d] float32/float16/bfloat16")
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (B, H)):
        raise ValueError("lse must be float32 [B,H]")
    st = load().fd_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, H, N, d,
                                  DTYPE_CODE[q.dtype], int(num_splits), float(scale), _ptr(out),
                                  DTYPE_CODE[out.dtype], _ptr(lse), _stream(q, stream))
    _check(st, "fd_decode_noalloc")
    return out, lse


def decode_paged(q, k_pages, v_pages, block_table, seqlens, num_splits=0, scale=None,
                 out_dtype=None, out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """fd_decode over a paged KV cache (fd_decode_paged).  Returns ``(out, lse)``.

    q [B,H,d]; k_pages/v_pages [num_pages, H, page_size, d]; block_table
    [B, max_pages] int32; seqlens [B] int32 (required).
    """
    _need_cuda(q, k_pages, v_pages, block_table, seqlens)
    if q.dtype not in DTYPE_CODE or k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise ValueError("q, K, V must share one dtype among float32/float16/bfloat16")
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages/v_pages must be [num_pages, H, page_size, d]")
    num_pages, H, page_size, d = k_pages.shape
    B = q.shape[0]
    if q.shape != (B, H, d):
        raise ValueError("q must be [B,H,d] with H, d of the pages")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be int32 [B, max_pages]")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    max_pages = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, H, d), dtype=odt, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    _need_cuda(out, lse)
    lib = load()
    need = lib.fd_workspace_size(B, H, max_pages * page_size, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    st = lib.fd_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seqlens),
                             B, H, d, page_size, max_pages, num_pages, DTYPE_CODE[q.dtype],
                             int(num_splits), float(scale), _ptr(out), DTYPE_CODE[out.dtype],
                             _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(q, stream))
    _check(st, "fd_decode_paged")
    return out, lse


def decode_gqa(q, k, v, seqlens=None, num_splits=0, scale=None, out_dtype=None, out=None,
               lse=None, return_lse=True, workspace=None, stream=None):
    """Grouped-query decode (fd_decode_gqa).  Returns ``(out, lse)``.

    q [B, Hq, d]; k, v [B, Hkv, N, d] with Hq a multiple of Hkv.
    """
    _need_cuda(q, k, v, seqlens)
    if q.dtype not in DTYPE_CODE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, K, V must share one dtype among float32/float16/bfloat16")
    if k.dim() != 4 or v.shape != k.shape or q.dim() != 3 or q.shape[0] != k.shape[0] \
            or q.shape[2] != k.shape[3] or q.shape[1] % k.shape[1]:
        raise ValueError("shapes: q [B,Hq,d], k/v [B,Hkv,N,d], Hq % Hkv == 0")
    B, Hkv, N, d = k.shape
    Hq = q.shape[1]
    if seqlens is not None and (seqlens.dtype != torch.int32 or seqlens.shape != (B,)):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, d), dtype=odt, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _need_cuda(out, lse)
    lib = load()
    need = lib.fd_workspace_size_gqa(B, Hq, Hkv, N, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    st = lib.fd_decode_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, Hq, Hkv, N, d,
                           DTYPE_CODE[q.dtype], int(num_splits), float(scale), _ptr(out),
                           DTYPE_CODE[out.dtype], _ptr(lse), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(q, stream))
    _check(st, "fd_decode_gqa")
    return out, lse



def decode_gqa_paged(q, k_pages, v_pages, block_table, seqlens, num_splits=0, scale=None,
                     out_dtype=None, out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """Grouped-query decode over a paged KV cache (fd_decode_gqa_paged).
    Returns ``(out, lse)``.

    q [B, Hq, d]; k_pages/v_pages [num_pages, Hkv, page_size, d] with Hq a
    multiple of Hkv and page_size 16 or a multiple of 32; block_table [B,
    max_pages] int32; seqlens [B] int32 (required).
    """
    _need_cuda(q, k_pages, v_pages, block_table, seqlens)
    if q.dtype not in DTYPE_CODE or k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise ValueError("q, K, V must share one dtype among float32/float16/bfloat16")
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page_size, d = k_pages.shape
    B, Hq = q.shape[0], q.shape[1]
    if q.dim() != 3 or q.shape[2] != d or Hq % Hkv:
        raise ValueError("q must be [B, Hq, d] with Hq a multiple of the pages' Hkv")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be int32 [B, max_pages]")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    max_pages = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, d), dtype=odt, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _need_cuda(out, lse)
    lib = load()
    need = lib.fd_workspace_size_gqa(B, Hq, Hkv, max_pages * page_size, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    st = lib.fd_decode_gqa_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                 _ptr(seqlens), B, Hq, Hkv, d, page_size, max_pages, num_pages,
                                 DTYPE_CODE[q.dtype], int(num_splits), float(scale), _ptr(out),
                                 DTYPE_CODE[out.dtype], _ptr(lse), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(q, stream))
    _check(st, "fd_decode_gqa_paged")
    return out, lse


def workspace_size_gqa(B, Hq, Hkv, N, d, num_splits=0) -> int:
    return load().fd_workspace_size_gqa(B, Hq, Hkv, N, d, num_splits)


def decode_fp8(q, k, v, k_scale, v_scale, seqlens=None, num_splits=0, scale=None, out_dtype=None,
               out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """fd_decode over an E4M3 KV cache with per-(b,h) scales (fd_decode_fp8).

    k, v: [B,H,N,d] torch.float8_e4m3fn (or uint8 holding E4M3 bytes);
    k_scale, v_scale: float32 [B,H]; q: float32/float16/bfloat16 [B,H,d].
    Returns ``(out, lse)``.
    """
    _need_cuda(q, k, v, k_scale, v_scale, seqlens)
    if q.dtype not in DTYPE_CODE:
        raise ValueError("q must be float32, float16 or bfloat16")
    if k.dtype not in (torch.float8_e4m3fn, torch.uint8) or v.dtype != k.dtype:
        raise ValueError("k, v must be float8_e4m3fn (or uint8 E4M3 bytes)")
    if k.dim() != 4 or v.shape != k.shape or q.shape != (k.shape[0], k.shape[1], k.shape[3]):
        raise ValueError("shapes: q [B,H,d], k/v [B,H,N,d]")
    B, H, N, d = k.shape
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != (B, H):
            raise ValueError("k_scale/v_scale must be float32 [B,H]")
    if seqlens is not None and (seqlens.dtype != torch.int32 or seqlens.shape != (B,)):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, H, d), dtype=odt, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    _need_cuda(out, lse)
    lib = load()
    need = lib.fd_workspace_size(B, H, N, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    st = lib.fd_decode_fp8(_ptr(q), DTYPE_CODE[q.dtype], _ptr(k), _ptr(v), _ptr(k_scale),
                           _ptr(v_scale), _ptr(seqlens), B, H, N, d, int(num_splits), float(scale),
                           _ptr(out), DTYPE_CODE[out.dtype], _ptr(lse), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(q, stream))
    _check(st, "fd_decode_fp8")
    return out, lse



def decode_gqa_fp8(q, k, v, k_scale, v_scale, seqlens=None, num_splits=0, scale=None, out_dtype=None,
                   out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """Grouped-query decode over an E4M3 KV cache (fd_decode_gqa_fp8).

    q: float32/float16/bfloat16 [B, Hq, d]; k, v: [B, Hkv, N, d]
    torch.float8_e4m3fn (or uint8 E4M3 bytes) with Hq a multiple of Hkv, d
    64, 128 or 256; k_scale, v_scale: float32 [B, Hkv].  Returns ``(out, lse)``.
    """
    _need_cuda(q, k, v, k_scale, v_scale, seqlens)
    if q.dtype not in DTYPE_CODE:
        raise ValueError("q must be float32, float16 or bfloat16")
    if k.dtype not in (torch.float8_e4m3fn, torch.uint8) or v.dtype != k.dtype:
        raise ValueError("k, v must be float8_e4m3fn (or uint8 E4M3 bytes)")
    if k.dim() != 4 or v.shape != k.shape or q.dim() != 3 or q.shape[0] != k.shape[0] \
            or q.shape[2] != k.shape[3] or q.shape[1] % k.shape[1]:
        raise ValueError("shapes: q [B,Hq,d], k/v [B,Hkv,N,d], Hq % Hkv == 0")
    B, Hkv, N, d = k.shape
    Hq = q.shape[1]
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != (B, Hkv):
            raise ValueError("k_scale/v_scale must be float32 [B,Hkv]")
    if seqlens is not None and (seqlens.dtype != torch.int32 or seqlens.shape != (B,)):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, d), dtype=odt, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _need_cuda(out, lse)
    lib = load()
    need = lib.fd_workspace_size_gqa(B, Hq, Hkv, N, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    st = lib.fd_decode_gqa_fp8(_ptr(q), DTYPE_CODE[q.dtype], _ptr(k), _ptr(v), _ptr(k_scale),
                               _ptr(v_scale), _ptr(seqlens), B, Hq, Hkv, N, d, int(num_splits),
                               float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(lse),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(q, stream))
    _check(st, "fd_decode_gqa_fp8")
    return out, lse



def decode_gqa_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens, num_splits=0,
                         scale=None, out_dtype=None, out=None, lse=None, return_lse=True, workspace=None,
                         stream=None):
    """Grouped-query decode over a paged E4M3 KV cache (fd_decode_gqa_paged_fp8).

    q: float32/float16/bfloat16 [B, Hq, d]; k_pages/v_pages [num_pages, Hkv,
    page_size, d] torch.float8_e4m3fn (or uint8 E4M3 bytes), d 64, 128 or
    256, page_size 16 or a multiple of 32; k_scale, v_scale float32 [B, Hkv]; block_table int32
    [B, max_pages]; seqlens int32 [B].  Returns ``(out, lse)``.
    """
    _need_cuda(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens)
    if q.dtype not in DTYPE_CODE:
        raise ValueError("q must be float32, float16 or bfloat16")
    if k_pages.dtype not in (torch.float8_e4m3fn, torch.uint8) or v_pages.dtype != k_pages.dtype:
        raise ValueError("pages must be float8_e4m3fn (or uint8 E4M3 bytes)")
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page_size, d = k_pages.shape
    B, Hq = q.shape[0], q.shape[1]
    if q.dim() != 3 or q.shape[2] != d or Hq % Hkv:
        raise ValueError("q must be [B, Hq, d] with Hq a multiple of the pages' Hkv")
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != (B, Hkv):
            raise ValueError("k_scale/v_scale must be float32 [B,Hkv]")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be int32 [B, max_pages]")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    max_pages = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    odt = out_dtype or q.dtype
    if out is None:
        out = torch.empty((B, Hq, d), dtype=odt, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _need_cuda(out, lse)
    lib = load()
    need = lib.fd_workspace_size_gqa(B, Hq, Hkv, max_pages * page_size, d, int(num_splits))
    if workspace is None:
        workspace = _cached_workspace(q.device, need)
    st = lib.fd_decode_gqa_paged_fp8(_ptr(q), DTYPE_CODE[q.dtype], _ptr(k_pages), _ptr(v_pages),
                                     _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(seqlens), B, Hq,
                                     Hkv, d, page_size, max_pages, num_pages, int(num_splits), float(scale),
                                     _ptr(out), DTYPE_CODE[out.dtype], _ptr(lse), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(q, stream))
    _check(st, "fd_decode_gqa_paged_fp8")
    return out, lse


def _one_device(*ts):
    """The index of the CUDA device that all given tensors are on."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device" if t.is_cuda else
                             "all tensors must be CUDA tensors (the library has no CPU path)")
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors (the library has no CPU path)")
    return dev


def _call(what, dev, stream, *args):
    """The library's call ``what`` with device ``dev`` current, on ``stream``
    (default: the device's current one)."""
    fn = getattr(_lib or load(), what)
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != FD_OK:
        raise FDError(st, what)


def _address(t):
    return None if t is None else t.data_ptr()


def _empty(stream, *args, **kw):
    """torch.empty for a call on ``stream``: memory of that stream's, since
    the current one may still work on what it gave back last; and kept until
    the current one, which will read the result, is done with it."""
    if stream is None:
        return torch.empty(*args, **kw)
    reader = torch.cuda.current_stream(kw["device"])
    with torch.cuda.stream(stream):
        t = torch.empty(*args, **kw)
    t.record_stream(reader)
    return t


def _rows(t, name):
    """Elements between the tokens of a packed [T, H, d] tensor whose tokens
    are contiguous (a view of a fused projection has them further apart)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, d]")
    T, H, d = t.shape
    if t.is_contiguous():
        return H * d
    far, head, one = t.stride()
    row = H * d
    if T == 0 or row == 0:
        return row
    if (d > 1 and one != 1) or (H > 1 and head != d):
        raise ValueError(f"{name}: the H*d elements of a token must be contiguous")
    if T == 1:
        return row
    if far < row:
        raise ValueError(f"{name}: tokens must not overlap")
    return far


def _int32(t, shape, name):
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)}")
    if t.numel() > INT_MAX and max(shape) > INT_MAX:   # the C call's sizes are ints, and ctypes cuts what passes them
        raise ValueError(f"{name}: sizes must be below 2^31")


def _whole(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors but packed rows must be contiguous")


def resize_pages(seqlens, target, block_table, free_pages, free_count, page_size, slots=None, positions=None,
                 cu_new=None, stream=None):
    """Every sequence of a paged cache to its target length, in place
    (fd_resize_pages): pages are taken from and given back to the stack
    ``free_pages[:free_count]``.

    seqlens, target int32 [B]; block_table int32 [B, max_pages]; free_pages
    int32 [num_pages]; free_count int32 [1]; slots and positions int32
    [max_tokens] receive the new tokens' places in the pool and positions
    (-1 and 0 behind the last), cu_new int32 [B+1] the offsets of the
    sequences' new tokens (allocated if only slots or positions are given).
    Returns ``cu_new``.  A sequence that could not grow keeps its length, and
    so do those behind it whose pages would only be free without it: running
    sequences go ahead of admissions.  Beams that share pages grow here, but are
    ended by ``reorder_pages`` (negative parents): shrinking them would give a
    shared page back once for each.
    """
    dev = _one_device(seqlens, target, block_table, free_pages, free_count, slots, positions, cu_new)
    if seqlens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("seqlens [B], block_table [B, max_pages], free_pages [num_pages]")
    B = seqlens.shape[0]
    width, pool, room = block_table.shape[1], free_pages.shape[0], 0
    if abs(page_size) > INT_MAX:
        raise ValueError("page_size must be below 2^31")
    _int32(seqlens, (B,), "seqlens")
    _int32(target, (B,), "target")
    _int32(block_table, (B, width), "block_table")
    _int32(free_pages, (pool,), "free_pages")
    _int32(free_count, (1,), "free_count")
    if slots is not None or positions is not None:
        room = (positions if slots is None else slots).numel()
        for t, n in ((slots, "slots"), (positions, "positions")):
            if t is not None:
                _int32(t, (room,), n)
        if cu_new is None:
            cu_new = _empty(stream, B + 1, dtype=torch.int32, device=seqlens.device)
    if cu_new is not None:
        _int32(cu_new, (B + 1,), "cu_new")
    _call("fd_resize_pages", dev, stream, seqlens.data_ptr(), target.data_ptr(), B, block_table.data_ptr(), width,
          free_pages.data_ptr(), free_count.data_ptr(), pool, page_size, _address(slots), _address(positions), room,
          _address(cu_new))
    return cu_new


def _append_args(k, v, slots, k_pages, v_pages):
    k_stride, v_stride = _rows(k, "k"), _rows(v, "v")
    if v.shape != k.shape or v.dtype != k.dtype or k.dtype not in DTYPE_CODE:
        raise ValueError("k and v must share one shape and dtype among float32/float16/bfloat16")
    T, H, d = k.shape
    _int32(slots, (T,), "slots")
    _whole(k_pages, v_pages)
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype != k_pages.dtype or shape[1] != H or shape[3] != d:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d] with Hkv, d of k")
    return T, H, d, k_stride, v_stride, DTYPE_CODE[k.dtype], k_pages.data_ptr(), v_pages.data_ptr(), shape[2], shape[0]


def append_paged(k, v, slots, k_pages, v_pages, stream=None):
    """New K and V rows into a paged cache, in place (fd_append_paged).

    k, v [T, Hkv, d] (a token's heads contiguous, tokens any multiple of 16
    bytes apart); slots int32 [T], negative ones skipped; k_pages/v_pages
    [num_pages, Hkv, page_size, d] of k's dtype.
    """
    dev = _one_device(k, v, slots, k_pages, v_pages)
    args = _append_args(k, v, slots, k_pages, v_pages)
    if k_pages.dtype != k.dtype:
        raise ValueError("the pages must have k's dtype")
    _call("fd_append_paged", dev, stream, k.data_ptr(), v.data_ptr(), slots.data_ptr(), *args)


def _scales(k_scale, v_scale, shape):
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
            raise ValueError("k_scale/v_scale must be contiguous float32 [B, Hkv]")


def append_paged_fp8(k, v, k_scale, v_scale, cu_new, slots, k_pages, v_pages, stream=None):
    """New K and V rows into E4M3 pages, in place (fd_append_paged_fp8): each
    row divided by its sequence's and head's scale and rounded to E4M3.

    k, v, slots as in append_paged; k_scale, v_scale float32 [B, Hkv]; cu_new
    int32 [B+1]; pages torch.float8_e4m3fn (or uint8 E4M3 bytes).
    """
    dev = _one_device(k, v, k_scale, v_scale, cu_new, slots, k_pages, v_pages)
    args = _append_args(k, v, slots, k_pages, v_pages)
    if k_pages.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError("pages must be float8_e4m3fn (or uint8 E4M3 bytes)")
    B = cu_new.numel() - 1
    _scales(k_scale, v_scale, (B, args[1]))
    _int32(cu_new, (B + 1,), "cu_new")
    _call("fd_append_paged_fp8", dev, stream, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
          cu_new.data_ptr(), slots.data_ptr(), B, *args)


def _rope_args(k, v, slots, positions, rope, k_pages, v_pages, q, q_out, interleaved, stream):
    """The arguments of the rotating appends from the positions on, and
    q_out, checked or allocated.  (In one piece: the call is short, and every
    further function shows in it.)"""
    k_stride, v_stride = _rows(k, "k"), _rows(v, "v")
    T, H, d = k.shape
    kind = k.dtype
    if v.shape != k.shape or v.dtype != kind or kind not in DTYPE_CODE:
        raise ValueError("k and v must share one shape and dtype among float32/float16/bfloat16")
    _int32(slots, (T,), "slots")
    _int32(positions, (T,), "positions")
    pages = k_pages.shape
    if len(pages) != 4 or v_pages.shape != pages or v_pages.dtype != k_pages.dtype or pages[1] != H or pages[3] != d:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d] with Hkv, d of k")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("all tensors but packed rows must be contiguous")
    table = rope.shape
    if len(table) != 2 or rope.dtype != torch.float32 or not rope.is_contiguous():
        raise ValueError("rope must be contiguous float32 [max_position, rot]: cosines, then sines")
    far, rot = table
    if far > INT_MAX or rot > INT_MAX:
        raise ValueError("rope: sizes must be below 2^31")
    Hq, q_stride, out_stride, q_at, out_at = 0, 0, 0, None, None
    if q is not None:
        q_stride = _rows(q, "q")
        rows, Hq, dq = q.shape
        if q.dtype != kind or rows != T or dq != d:
            raise ValueError("q must be [T, Hq, d] of k's tokens, head dim and dtype")
        if q_out is None:
            q_out, out_stride = _empty(stream, q.shape, dtype=kind, device=q.device), Hq * d
        elif q_out.shape != q.shape or q_out.dtype != kind:
            raise ValueError("q_out must have q's shape and dtype")
        else:
            out_stride = _rows(q_out, "q_out")
        if Hq:
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    return ((q_at, k.data_ptr(), v.data_ptr()),
            (slots.data_ptr(), positions.data_ptr(), rope.data_ptr(), far, rot, bool(interleaved)),
            (T, Hq, H, d, q_stride, k_stride, v_stride, DTYPE_CODE[kind], out_at, out_stride, k_pages.data_ptr(),
             v_pages.data_ptr(), pages[2], pages[0]), q_out)


def append_rope_paged(k, v, slots, positions, rope, k_pages, v_pages, q=None, q_out=None, interleaved=False, stream=None):
    """New K and V rows into a paged cache, in place, K rotated by its position
    on the way, and q beside it (fd_append_rope_paged).  Returns the rotated
    q, or None without q.

    k, v, slots, pages as in append_paged; positions int32 [T]; rope float32
    [max_position, rot], a row the cosines of rot/2 angles and then their
    sines; the pairs are elements i and i + rot/2 of a head, or 2i and 2i + 1
    with ``interleaved``.  q [T, Hq, d] of k's dtype; q_out [T, Hq, d] may be q.
    Tokens with a negative slot are skipped, their rows of q_out too.
    """
    dev = _one_device(k, v, slots, positions, rope, k_pages, v_pages, q, q_out)
    rows, where, sizes, q_out = _rope_args(k, v, slots, positions, rope, k_pages, v_pages, q, q_out, interleaved, stream)
    if k_pages.dtype != k.dtype:
        raise ValueError("the pages must have k's dtype")
    _call("fd_append_rope_paged", dev, stream, *rows, *where, *sizes)
    return q_out


def append_rope_paged_fp8(k, v, k_scale, v_scale, cu_new, slots, positions, rope, k_pages, v_pages, q=None, q_out=None,
                          interleaved=False, stream=None):
    """append_rope_paged into E4M3 pages (fd_append_rope_paged_fp8): k_scale,
    v_scale float32 [B, Hkv] and cu_new int32 [B+1] as in append_paged_fp8.
    Returns the rotated q, or None without q."""
    dev = _one_device(k, v, k_scale, v_scale, cu_new, slots, positions, rope, k_pages, v_pages, q, q_out)
    rows, where, sizes, q_out = _rope_args(k, v, slots, positions, rope, k_pages, v_pages, q, q_out, interleaved, stream)
    if k_pages.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError("pages must be float8_e4m3fn (or uint8 E4M3 bytes)")
    B = cu_new.numel() - 1
    _scales(k_scale, v_scale, (B, sizes[2]))
    _int32(cu_new, (B + 1,), "cu_new")
    _call("fd_append_rope_paged_fp8", dev, stream, *rows, k_scale.data_ptr(), v_scale.data_ptr(), cu_new.data_ptr(),
          *where, B, *sizes)
    return q_out


def workspace_size_extend(B, total_q, Hq, Hkv, d) -> int:
    """Bytes of workspace prefill, extend_paged and extend_paged_fp8 need."""
    return load().fd_workspace_size_extend(B, total_q, Hq, Hkv, d)


@functools.lru_cache(maxsize=1024)
def _known_extend_bytes(dev, *sizes):
    with torch.cuda.device(dev):
        n = workspace_size_extend(*sizes)
    if n == 0:   # an exception is not remembered: a CUDA error may be over by the next call
        raise LookupError
    return n


def _extend_bytes(dev, *sizes):
    """workspace_size_extend on a device, which depends on nothing else; some
    bytes where it gives none, so that the call itself says why."""
    try:
        return _known_extend_bytes(dev, *sizes)
    except LookupError:
        return 256


def _extend_out(dev, q, B, Hkv, out_dtype, out, lse, return_lse, workspace, stream):
    """out, lse and the workspace of the attention calls of several new
    tokens, checked or allocated (the workspace for this one call)."""
    shape = T, Hq, d = q.shape
    where = q.device
    if out is None:
        out = _empty(stream, shape, dtype=out_dtype or q.dtype, device=where)
    elif out.shape != shape or out.get_device() != dev or not out.is_contiguous():
        raise ValueError("out must be contiguous [T, Hq, d] on q's device")
    if out.dtype not in DTYPE_CODE:
        raise ValueError("out must be float32/float16/bfloat16")
    if lse is not None:
        if lse.dtype != torch.float32 or lse.shape != (T, Hq) or lse.get_device() != dev or not lse.is_contiguous():
            raise ValueError("lse must be contiguous float32 [T, Hq] on q's device")
    elif return_lse:
        lse = _empty(stream, (T, Hq), dtype=torch.float32, device=where)
    if workspace is None:
        workspace = _empty(stream, _extend_bytes(dev, B, T, Hq, Hkv, d), dtype=torch.uint8, device=where)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on q's device")
    return out, lse, workspace


def _tail(d, scale, out, lse, workspace):
    """The arguments that the attention calls of several new tokens end with."""
    return (1.0 / math.sqrt(d) if scale is None else scale, out.data_ptr(), DTYPE_CODE[out.dtype], _address(lse),
            workspace.data_ptr(), workspace.numel() * workspace.element_size())


def prefill(q, k, v, cu_seqlens_q, cu_seqlens_k=None, causal=True, scale=None, out_dtype=None, out=None, lse=None,
            return_lse=True, workspace=None, stream=None):
    """Attention over packed prompts (fd_prefill).  Returns ``(out, lse)``.

    q [Tq, Hq, d], k, v [Tk, Hkv, d] float16 or bfloat16, Hq a multiple of
    Hkv, d 64 or 128; a token's heads contiguous, tokens any multiple of 16
    bytes apart.  Sequence b's rows are cu_seqlens_q[b] ..
    cu_seqlens_q[b+1]-1 of q, and the same of cu_seqlens_k (default: the same
    offsets) of k and v; with ``causal`` the last query sees all keys, the
    one before all but the last, and so on.  out [Tq, Hq, d], lse [Tq, Hq]
    float32; rows outside the sequences are not written.
    """
    cu_k = cu_seqlens_q if cu_seqlens_k is None else cu_seqlens_k
    dev = _one_device(q, k, v, cu_seqlens_q, cu_k)
    q_stride, k_stride, v_stride = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    if q.dtype not in (torch.float16, torch.bfloat16) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype, float16 or bfloat16")
    (T, Hq, d), (Tk, Hkv, dk) = q.shape, k.shape
    if v.shape != k.shape or dk != d or Hkv == 0 or Hq % Hkv:
        raise ValueError("shapes: q [Tq, Hq, d], k/v [Tk, Hkv, d], Hq % Hkv == 0")
    if cu_seqlens_k is None and Tk != T:
        raise ValueError("without cu_seqlens_k, k and v must have q's tokens")
    B = cu_seqlens_q.numel() - 1
    _int32(cu_seqlens_q, (B + 1,), "cu_seqlens_q")
    _int32(cu_k, (B + 1,), "cu_seqlens_k")
    out, lse, workspace = _extend_out(dev, q, B, Hkv, out_dtype, out, lse, return_lse, workspace, stream)
    _call("fd_prefill", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(),
          cu_k.data_ptr(), B, T, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, DTYPE_CODE[q.dtype], bool(causal),
          *_tail(d, scale, out, lse, workspace))
    return out, lse


def _extend_args(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens):
    q_stride = _rows(q, "q")
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("q must be float16 or bfloat16")
    _whole(k_pages, v_pages)
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d]")
    (num_pages, Hkv, page_size, dk), (T, Hq, d) = k_pages.shape, q.shape
    if dk != d or Hkv == 0 or Hq % Hkv:
        raise ValueError("q must be [T, Hq, d] with Hq a multiple of the pages' Hkv")
    B = seqlens.numel()
    _int32(seqlens, (B,), "seqlens")
    _int32(cu_seqlens_q, (B + 1,), "cu_seqlens_q")
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, max_pages]")
    width = block_table.shape[1]
    _int32(block_table, (B, width), "block_table")
    return B, T, Hq, Hkv, d, q_stride, page_size, width, num_pages


def extend_paged(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, scale=None, out_dtype=None, out=None,
                 lse=None, return_lse=True, workspace=None, stream=None):
    """Attention of new tokens over a paged cache that holds them already
    (fd_extend_paged).  Returns ``(out, lse)``.

    q [T, Hq, d] float16 or bfloat16, sequence b's new tokens at rows
    cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1; k_pages/v_pages [num_pages, Hkv,
    page_size, d] of q's dtype, page_size a multiple of 16; block_table int32
    [B, max_pages]; seqlens int32 [B], the new tokens included.  A
    sequence's last new token sees all seqlens[b] tokens, the one before all
    but the last, and so on.
    """
    dev = _one_device(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens)
    args = _extend_args(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens)
    if k_pages.dtype != q.dtype:
        raise ValueError("the pages must have q's dtype")
    out, lse, workspace = _extend_out(dev, q, args[0], args[3], out_dtype, out, lse, return_lse, workspace, stream)
    _call("fd_extend_paged", dev, stream, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
          block_table.data_ptr(), cu_seqlens_q.data_ptr(), seqlens.data_ptr(), *args, DTYPE_CODE[q.dtype],
          *_tail(args[4], scale, out, lse, workspace))
    return out, lse


def extend_paged_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_seqlens_q, seqlens, scale=None,
                     out_dtype=None, out=None, lse=None, return_lse=True, workspace=None, stream=None):
    """extend_paged over E4M3 pages (fd_extend_paged_fp8): pages
    torch.float8_e4m3fn (or uint8 E4M3 bytes), k_scale, v_scale float32
    [B, Hkv].  Returns ``(out, lse)``."""
    dev = _one_device(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_seqlens_q, seqlens)
    args = _extend_args(q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens)
    if k_pages.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError("pages must be float8_e4m3fn (or uint8 E4M3 bytes)")
    _scales(k_scale, v_scale, (args[0], args[3]))
    out, lse, workspace = _extend_out(dev, q, args[0], args[3], out_dtype, out, lse, return_lse, workspace, stream)
    _call("fd_extend_paged_fp8", dev, stream, q.data_ptr(), DTYPE_CODE[q.dtype], k_pages.data_ptr(),
          v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), cu_seqlens_q.data_ptr(),
          seqlens.data_ptr(), *args, *_tail(args[4], scale, out, lse, workspace))
    return out, lse


def workspace_size_beam(R, W, V, K) -> int:
    """Bytes of workspace beam_select needs."""
    return load().fd_workspace_size_beam(R, W, V, K)


@functools.lru_cache(maxsize=1024)
def _known_beam_bytes(dev, *sizes):
    with torch.cuda.device(dev):
        n = workspace_size_beam(*sizes)
    if n == 0:   # as in _known_extend_bytes
        raise LookupError
    return n


def beam_select(logits, scores, num=None, finished=None, eos=-1, workspace=None, stream=None):
    """Beam search's selection (fd_beam_select): of the W * V continuations of
    each request's W beams the ``num`` (default W) with the largest score, the
    best first.  Returns ``(scores, parents, tokens, finished)``, [R, num]
    float32, int32, int32 and bool.

    logits [R, W, V] float32, float16 or bfloat16, a beam's V neighbouring (any
    strides else); scores float32 [R, W]; finished bool [R, W]: beams that go
    on with ``eos`` alone at the score they have, their logits not read.
    Equal scores in order of beam and token.  Where a request has fewer
    continuations (of -inf, NaN and beams without a finite score there are
    none) the rest is -inf, -1, -1 and finished.  A beam's scores share the
    error of a float32 sum, below 1e-5 (some 2e-7 on ordinary rows), whose last
    bits follow the batch's size and the rows' alignment.
    """
    dev = _one_device(logits, scores, finished)
    if logits.dim() != 3 or logits.dtype not in DTYPE_CODE:
        raise ValueError("logits must be [R, W, V] float32/float16/bfloat16")
    (R, W, V), (far, near, one) = logits.shape, logits.stride()
    if V > 1 and one != 1:
        raise ValueError("logits: a beam's V must be contiguous")
    if R > INT_MAX or W > INT_MAX or V > INT_MAX:
        raise ValueError("logits: sizes must be below 2^31")
    if scores.dtype != torch.float32 or scores.shape != (R, W) or not scores.is_contiguous():
        raise ValueError("scores must be contiguous float32 [R, W]")
    if finished is not None and (finished.dtype != torch.bool or finished.shape != (R, W) or not finished.is_contiguous()):
        raise ValueError("finished must be contiguous bool [R, W]")
    K = W if num is None else num
    if not 1 <= K <= INT_MAX:
        raise ValueError("num must be positive")
    if not -1 <= eos < max(V, 1):
        raise ValueError("eos must be a token, or -1")
    where = logits.device
    empty = torch.empty if stream is None else functools.partial(_empty, stream)
    if workspace is None:
        try:
            n = _known_beam_bytes(dev, R, W, V, K)
        except LookupError:
            n = 256   # the call itself says why
        workspace = empty(n, dtype=torch.uint8, device=where)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the logits' device")
    shape = (R, K)
    out = empty(shape, dtype=torch.float32, device=where)
    parents = empty(shape, dtype=torch.int32, device=where)
    tokens = empty(shape, dtype=torch.int32, device=where)
    over = empty(shape, dtype=torch.bool, device=where)
    _call("fd_beam_select", dev, stream, logits.data_ptr(), DTYPE_CODE[logits.dtype], far, near, scores.data_ptr(),
          _address(finished), R, W, V, K, eos, out.data_ptr(), parents.data_ptr(), tokens.data_ptr(), over.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, parents, tokens, over


def workspace_size_reorder(R, W, max_pages) -> int:
    """Bytes of workspace reorder_pages needs."""
    return load().fd_workspace_size_reorder(R, W, max_pages)


_known_reorder_bytes = functools.lru_cache(maxsize=1024)(workspace_size_reorder)   # (of the sizes alone)


def reorder_pages(parents, seqlens, block_table, free_pages, free_count, page_size, copies=None, granted=None, workspace=None,
                  stream=None):
    """The beams' cached states to those of their parents, in place
    (fd_reorder_pages).  Returns ``(copies, granted)``; ``copy_pages`` has to
    make the copies in each layer's pages.

    parents int32 [R, W]: of every beam the beam of its request that it goes on
    from, negative where it ends.  Beam w of request r is sequence r*W + w:
    seqlens int32 [R*W] (or [R, W]); block_table int32 [R*W, max_pages];
    free_pages int32 [num_pages] and free_count int32 [1], the stack of
    resize_pages.  copies int32 [R*W, 3]: page from, page to and rows, -1, -1
    and 0 without a copy; granted int32 [R]: 0 where pages were missing and the
    request stays as it was, so that its old scores, flags and logits hold on and
    the choice is made again in a later step.
    """
    dev = _one_device(parents, seqlens, block_table, free_pages, free_count, copies, granted)
    if parents.dim() != 2 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("parents [R, W], block_table [R*W, max_pages], free_pages [num_pages]")
    R, W = parents.shape
    B, width, pool = R * W, block_table.shape[1], free_pages.shape[0]
    if abs(page_size) > INT_MAX:
        raise ValueError("page_size must be below 2^31")
    _int32(parents, (R, W), "parents")
    _int32(seqlens, (R, W) if seqlens.dim() == 2 else (B,), "seqlens")
    _int32(block_table, (B, width), "block_table")
    _int32(free_pages, (pool,), "free_pages")
    _int32(free_count, (1,), "free_count")
    where = parents.device
    empty = torch.empty if stream is None else functools.partial(_empty, stream)
    if copies is None:
        copies = empty((B, 3), dtype=torch.int32, device=where)
    else:
        _int32(copies, (B, 3), "copies")
    if granted is None:
        granted = empty(R, dtype=torch.int32, device=where)
    else:
        _int32(granted, (R,), "granted")
    if workspace is None:
        workspace = empty(max(_known_reorder_bytes(R, W, width), 256), dtype=torch.uint8, device=where)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the parents' device")
    _call("fd_reorder_pages", dev, stream, parents.data_ptr(), R, W, seqlens.data_ptr(), block_table.data_ptr(), width,
          free_pages.data_ptr(), free_count.data_ptr(), pool, page_size, copies.data_ptr(), granted.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return copies, granted


def copy_pages(copies, k_pages, v_pages, stream=None):
    """Rows of pages to other pages, in place (fd_copy_pages): the copies that
    reorder_pages asks for, of one layer.

    copies int32 [n, 3]: page from, page to, rows; k_pages/v_pages [num_pages,
    Hkv, page_size, d] float32, float16, bfloat16 or float8_e4m3fn (or uint8
    E4M3 bytes).
    """
    dev = _one_device(copies, k_pages, v_pages)
    if copies.dim() != 2:
        raise ValueError("copies must be int32 [n, 3]")
    _int32(copies, (copies.shape[0], 3), "copies")
    _whole(k_pages, v_pages)
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages/v_pages must be [num_pages, Hkv, page_size, d]")
    kind = 3 if k_pages.dtype in (torch.float8_e4m3fn, torch.uint8) else DTYPE_CODE.get(k_pages.dtype)
    if kind is None:
        raise ValueError("pages must be float32/float16/bfloat16/float8_e4m3fn (or uint8 E4M3 bytes)")
    num_pages, Hkv, page_size, d = k_pages.shape
    if max(Hkv, page_size, d) > INT_MAX:
        raise ValueError("pages: sizes must be below 2^31")
    _call("fd_copy_pages", dev, stream, copies.data_ptr(), copies.shape[0], Hkv, d, kind, k_pages.data_ptr(),
          v_pages.data_ptr(), page_size, num_pages)


def decode_split(q, k, v, num_splits, seqlens=None, scale=None, stream=None, o_part=None,
                 m_part=None, l_part=None, lse_part=None):
    """Stage 1 alone (fd_decode_split).  Returns ``(o_part, m_part, l_part, lse_part)``.

    The partial buffers may be passed in (float32, [B,H,P,d] and [B,H,P]);
    those not given are allocated."""
    B, H, N, d = _check_qkv(q, k, v, seqlens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    P = int(num_splits)
    dev = q.device
    if o_part is None:
        o_part = torch.empty((B, H, P, d), dtype=torch.float32, device=dev)
    for t in (m_part, l_part, lse_part):
        if t is not None and (t.shape != (B, H, P) or t.dtype != torch.float32
                              or not t.is_contiguous()):
            raise ValueError("m_part / l_part / lse_part must be contiguous float32 [B,H,P]")
    if o_part.shape != (B, H, P, d) or o_part.dtype != torch.float32 or not o_part.is_contiguous():
        raise ValueError("o_part must be contiguous float32 [B,H,P,d]")
    if m_part is None:
        m_part = torch.empty((B, H, P), dtype=torch.float32, device=dev)
    if l_part is None:
        l_part = torch.empty((B, H, P), dtype=torch.float32, device=dev)
    if lse_part is None:
        lse_part = torch.empty((B, H, P), dtype=torch.float32, device=dev)
    _need_cuda(o_part, m_part, l_part, lse_part)
    st = load().fd_decode_split(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), B, H, N, d,
                                DTYPE_CODE[q.dtype], P, float(scale), _ptr(o_part), _ptr(m_part),
                                _ptr(l_part), _ptr(lse_part), _stream(q, stream))
    _check(st, "fd_decode_split")
    return o_part, m_part, l_part, lse_part


def _combine_out(o_part, out_dtype, out, lse, return_lse):
    B, H, P, d = o_part.shape
    if out is None:
        out = torch.empty((B, H, d), dtype=out_dtype or torch.float32, device=o_part.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=o_part.device)
    _need_cuda(out, lse)
    return B, H, P, d, out, lse


def combine_mlo(o_part, m_part, l_part, out_dtype=None, out=None, lse=None, return_lse=True,
                stream=None):
    """Stage 2, m/l/o merge (fd_combine_mlo).  Returns ``(out, lse)``."""
    _need_cuda(o_part, m_part, l_part)
    B, H, P, d, out, lse = _combine_out(o_part, out_dtype, out, lse, return_lse)
    for t in (o_part, m_part, l_part):
        if t.dtype != torch.float32:
            raise ValueError("partials must be float32")
    if m_part.shape != (B, H, P) or l_part.shape != (B, H, P):
        raise ValueError("m_part/l_part must be [B,H,P]")
    st = load().fd_combine_mlo(_ptr(o_part), _ptr(m_part), _ptr(l_part), B, H, P, d, _ptr(out),
                               DTYPE_CODE[out.dtype], _ptr(lse), _stream(o_part, stream))
    _check(st, "fd_combine_mlo")
    return out, lse


def combine_lse(o_part, lse_part, out_dtype=None, out=None, lse=None, return_lse=True,
                stream=None):
    """Stage 2, LSE merge (fd_combine_lse).  Returns ``(out, lse)``."""
    _need_cuda(o_part, lse_part)
    B, H, P, d, out, lse = _combine_out(o_part, out_dtype, out, lse, return_lse)
    for t in (o_part, lse_part):
        if t.dtype != torch.float32:
            raise ValueError("partials must be float32")
    if lse_part.shape != (B, H, P):
        raise ValueError("lse_part must be [B,H,P]")
    st = load().fd_combine_lse(_ptr(o_part), _ptr(lse_part), B, H, P, d, _ptr(out),
                               DTYPE_CODE[out.dtype], _ptr(lse), _stream(o_part, stream))
    _check(st, "fd_combine_lse")
    return out, lse


def merge_lse(o_a, lse_a, o_b, lse_b, out=None, lse=None, stream=None):
    """(o_a, lse_a) (+) (o_b, lse_b) row by row (fd_merge_lse).  Returns ``(out, lse)``.

    o_*: float32 [..., d]; lse_*: float32 [...] (same leading shape).  ``out``
    / ``lse`` may be ``o_a`` / ``lse_a`` for an in-place fold.
    """
    _need_cuda(o_a, lse_a, o_b, lse_b)
    for t in (o_a, lse_a, o_b, lse_b):
        if t.dtype != torch.float32:
            raise ValueError("partials must be float32")
    if o_b.shape != o_a.shape or lse_a.shape != o_a.shape[:-1] or lse_b.shape != lse_a.shape:
        raise ValueError("shapes: o [..., d], lse [...]")
    d = o_a.shape[-1]
    rows = lse_a.numel()
    if out is None:
        out = torch.empty_like(o_a)
    if lse is None:
        lse = torch.empty_like(lse_a)
    _need_cuda(out, lse)
    st = load().fd_merge_lse(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), rows, d, _ptr(out),
                             _ptr(lse), _stream(o_a, stream))
    _check(st, "fd_merge_lse")
    return out, lse


def selftest_wait_timeout(stream=None) -> None:
    """Launch the bounded-wait self-test (fd_selftest_wait_timeout): a kernel
    whose wait nothing completes gives up after the kernels' wait limit (1 s)
    and records FD_ERR_DEVICE_TIMEOUT, read back by device_status()."""
    s = stream if stream is not None else torch.cuda.current_stream()
    rc = load().fd_selftest_wait_timeout(ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise FDError(rc, "fd_selftest_wait_timeout")


def device_status(reset: bool = True) -> int:
    """FD_OK, or what a kernel recorded: FD_ERR_DEVICE_TIMEOUT, FD_ERR_BAD_PAGE,
    FD_ERR_BAD_OFFSETS or FD_ERR_BAD_INDEX (synchronises)."""
    return load().fd_device_status(1 if reset else 0)
