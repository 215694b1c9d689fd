"""Paged-KV attention with a learned relative-position bias for sm_103a GPUs.

The compute lives in libinkling_rel_attn.so (C ABI, include/inkling_rel_attn.h);
this package is its thin Python binding.  Importing the package does not load
the library; the first call does, and fails loudly if it was not built.
"""

from .ops import (  # noqa: F401
    InklingError,
    build_tables,
    choose_splits,
    compact_pages,
    copy_pages,
    decode,
    decode_inputs,
    decode_multi,
    decode_multi_workspace_bytes,
    decode_q4,
    decode_q4_workspace_bytes,
    decode_q8,
    decode_q8_workspace_bytes,
    decode_workspace_bytes,
    fork_pages,
    kv_append,
    kv_append_q4,
    kv_append_q8,
    kv_conv_append,
    kv_read_q4,
    kv_read_q8,
    prefill,
    prefill_inputs,
    prefill_q4,
    prefill_q4_workspace_bytes,
    prefill_q8,
    prefill_q8_workspace_bytes,
    release_pages,
)

__all__ = ["InklingError", "build_tables", "choose_splits", "compact_pages", "copy_pages", "decode",
           "decode_inputs", "decode_multi", "decode_multi_workspace_bytes", "decode_q4",
           "decode_q4_workspace_bytes", "decode_q8", "decode_q8_workspace_bytes", "decode_workspace_bytes",
           "fork_pages", "kv_append", "kv_append_q4", "kv_append_q8", "kv_conv_append", "kv_read_q4",
           "kv_read_q8", "prefill", "prefill_inputs", "prefill_q4", "prefill_q4_workspace_bytes",
           "prefill_q8", "prefill_q8_workspace_bytes", "release_pages"]
