"""Sizes at the ends of 32 bits in the calls around decode, without a GPU:
refused where an index could not hold them, by the library and by the
binding."""
import contextlib
import ctypes

import pytest
import torch

from split_kv_fd_gb300 import fd as fdmod

P = ctypes.c_void_p
X = P(4096)      # aligned, never dereferenced
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    return fdmod.load(build_if_missing=True)


def test_resize_counts_sequences_in_32_bits(lib):
    assert lib.fd_resize_pages(X, X, (1 << 30) + 1, X, 1, X, X, 9, 16, X, X, 8, X, None) == INVALID


def test_tensors_past_an_int_are_refused():
    """ctypes would cut the size: 2^32 + 5 slots would count as 5."""
    big = torch.empty((1 << 32) + 5, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError):
        fdmod._int32(big, tuple(big.shape), "slots")
    wide = torch.empty(1 << 10, 1 << 22, dtype=torch.int32, device="meta")   # 2^32 entries, but no size that large
    fdmod._int32(wide, tuple(wide.shape), "block_table")


@pytest.mark.parametrize("page_size", [1 << 31, (1 << 32) + 16, 16 - (1 << 32)])
def test_page_size_is_an_int(page_size, monkeypatch):
    monkeypatch.setattr(fdmod, "_one_device", lambda *ts: 0)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="page_size"):
        fdmod.resize_pages(i, i, i[:, None], i, i[:1], page_size)


@pytest.mark.parametrize("stride", [0, 1, -3, 12345, (1 << 44) + 1])
def test_one_token_has_no_stride(lib, stride):
    """Without heads, so that the calls end behind their checks of sizes."""
    for t in (0, 1):
        assert lib.fd_prefill(X, X, X, X, X, 2, t, t, 0, 2, 128, stride, stride, stride, 2, 1, 0.1, X, 2, None, None, 0, None) == 0
        assert lib.fd_extend_paged(X, X, X, X, X, X, 2, t, 0, 2, 128, stride, 64, 4, 9, 2, 0.1, X, 2, None, None, 0, None) == 0
        for dtype in (0, 1, 2):
            assert lib.fd_append_paged(X, X, X, t, 0, 128, stride, stride, dtype, X, X, 16, 9, None) == 0
            assert lib.fd_append_paged_fp8(X, X, X, X, X, X, 2, t, 0, 128, stride, stride, dtype, X, X, 16, 9, None) == 0


@pytest.mark.parametrize("stride", [-8, 1, 257, 260])
def test_several_tokens_have_one(lib, stride):
    assert lib.fd_prefill(X, X, X, X, X, 2, 2, 2, 2, 2, 128, stride, 256, 256, 2, 1, 0.1, X, 2, None, None, 0, None) == INVALID
    assert lib.fd_prefill(X, X, X, X, X, 2, 2, 2, 2, 2, 128, 256, 256, stride, 2, 1, 0.1, X, 2, None, None, 0, None) == INVALID
    assert lib.fd_append_paged(X, X, X, 2, 2, 128, 256, stride, 2, X, X, 16, 9, None) == INVALID
    if stride != 260:   # 1040 bytes of float32 are on the boundary
        assert lib.fd_append_paged(X, X, X, 2, 2, 128, stride, 256, 0, X, X, 16, 9, None) == INVALID


def test_keys_are_counted_in_32_bits(lib):
    """A block of keys behind the last one must fit an int.  (Without a
    workspace, so that no call that passes the checks is launched.)"""
    def extend(page, width):
        return lib.fd_extend_paged(X, X, X, X, X, X, 2, 4, 4, 2, 128, 512, page, width, 9, 2, 0.1, X, 2, None, None, 0, None)

    def prefill(tq, tk):
        return lib.fd_prefill(X, X, X, X, X, 2, tq, tk, 4, 2, 128, 512, 256, 256, 2, 1, 0.1, X, 2, None, None, 0, None)

    top = (1 << 31) - 1 - 256
    assert extend(16, (1 << 27) - 1) == INVALID and extend(128, (1 << 24) - 1) == INVALID
    assert extend(16, top // 16) != INVALID
    assert prefill(4, top + 1) == INVALID and prefill(top + 1, 4) == INVALID
    assert prefill(4, top) != INVALID


def test_sequences_are_counted_in_32_bits(lib):
    assert lib.fd_append_paged_fp8(X, X, X, X, X, X, (1 << 30) + 1, 2, 2, 128, 256, 256, 2, X, X, 16, 9, None) == INVALID
    assert lib.fd_workspace_size_extend((1 << 30) + 1, 1, 1, 1, 64) == 0
    assert lib.fd_workspace_size_extend(1 << 20, 1, 1 << 11, 1 << 11, 64) == 0


def test_a_failed_workspace_query_is_not_remembered(monkeypatch):
    """The query gives 0 on a CUDA error, or where the library has no such sizes."""
    answers = iter([0, 0, 4096, 8192])
    monkeypatch.setattr(fdmod, "workspace_size_extend", lambda *sizes: next(answers))
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    sizes = (0, 7, 7, 7, 7, 64)
    try:
        assert [fdmod._extend_bytes(*sizes) for _ in range(4)] == [256, 256, 4096, 4096]
    finally:
        for f in vars(fdmod).values():     # nothing made up stays for later calls
            if hasattr(f, "cache_clear"):
                f.cache_clear()
