"""libspecverify: the verify-and-sample step of speculative decoding on GB300.

The product is the C-ABI shared library built from ``csrc/`` (see
``include/specverify.h``); this package holds its build script, a thin ctypes
binding with the same entry-point names, and the seeded synthetic workloads
used by the tests and the benchmark.
"""
from ._lib import (FLAG_BAD_LENGTH, FLAG_BAD_PAGE, FLAG_BAD_TOKEN, FLAG_NONFINITE,
                   FLAG_RESIDUAL_FALLBACK, FLAG_TIMEOUT, FLAG_ZERO_MASS, KVCache, SpecVerifyError,
                   alloc_kv_cache, alloc_workspace, attention_workspace_bytes, library_path, load,
                   spec_chunk_attention, spec_kv_append, spec_kv_read, spec_lmhead_draft,
                   spec_lmhead_verify, spec_lmhead_verify_drafted, spec_verify,
                   spec_verify_greedy, spec_verify_probs, status_string, test_attention_stall,
                   test_lmhead_stall, workspace_bytes)

__all__ = ["spec_verify", "spec_verify_greedy", "spec_lmhead_verify", "spec_lmhead_draft",
           "spec_lmhead_verify_drafted", "spec_kv_append", "spec_kv_read", "spec_chunk_attention",
           "spec_verify_probs", "KVCache", "alloc_kv_cache", "attention_workspace_bytes",
           "workspace_bytes",
           "alloc_workspace", "load", "library_path", "status_string", "SpecVerifyError",
           "FLAG_ZERO_MASS", "FLAG_NONFINITE", "FLAG_RESIDUAL_FALLBACK", "FLAG_TIMEOUT",
           "FLAG_BAD_TOKEN", "FLAG_BAD_PAGE", "FLAG_BAD_LENGTH", "test_lmhead_stall", "test_attention_stall"]
