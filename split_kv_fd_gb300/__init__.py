"""split_kv_fd_gb300: split-KV decode attention (FlashDecoding) for GB300.

The compute path is the CUDA library ``libfd.so`` (C ABI in include/fd.h,
kernels in csrc/); ``fd`` is its Python binding.  ``workloads`` and
``inputs`` hold the synthetic workload shapes and the seeded input drawing.
"""
from .fd import (FDError, append_paged, append_paged_fp8, append_rope_paged, append_rope_paged_fp8,  # noqa: F401
                 auto_num_splits, beam_select, combine_lse, combine_mlo, copy_pages, decode, decode_fp8, decode_gqa,
                 decode_gqa_fp8, decode_gqa_paged, decode_gqa_paged_fp8, decode_noalloc, decode_paged, decode_split,
                 device_status, extend_paged, extend_paged_fp8, load, merge_lse, new_workspace, num_sms, prefill,
                 reorder_pages, resize_pages, selftest_wait_timeout, workspace_size, workspace_size_beam,
                 workspace_size_extend, workspace_size_gqa, workspace_size_reorder)

__all__ = ["FDError", "append_paged", "append_paged_fp8", "append_rope_paged", "append_rope_paged_fp8", "auto_num_splits",
           "beam_select", "combine_lse", "combine_mlo", "copy_pages", "decode", "decode_fp8", "decode_gqa", "decode_gqa_fp8",
           "decode_gqa_paged", "decode_gqa_paged_fp8", "decode_noalloc", "workspace_size_gqa", "decode_paged", "decode_split",
           "device_status", "extend_paged", "extend_paged_fp8", "load", "merge_lse", "new_workspace", "num_sms", "prefill",
           "reorder_pages", "resize_pages", "selftest_wait_timeout", "workspace_size", "workspace_size_beam",
           "workspace_size_extend", "workspace_size_reorder"]
