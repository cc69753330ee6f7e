"""Sizes at the ends of 32 bits in the calls around decode, without a GPU:
refused where an index could not hold them, by the library and by the
binding."""
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
