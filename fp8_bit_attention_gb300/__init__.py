"""ExpCast FP8 attention for GB300 (sm_103a).

The computation lives in libovc (CUDA, C ABI in include/ovc.h); this package
is its Python binding.  ``attention(q, k, v)`` is the full call.  Importing
the package does not load the library; the first call does, and fails loudly
if it has not been built.
"""
from .api import (CapturedAttention, OvcError, Prepared, Repair, attention, attention_prepared, attention_probe,
                  attention_v_repair, attention_workspace_bytes, attn_flags, group_v, device_status, flops, prepare, prepare_v_repair,
                  prepare_workspace_bytes, repair_workspace_bytes, baseline_attention)
from .paged import (KVCache, kv_cache, kv_cache_read, kv_cache_write, paged_attention, paged_attention_workspace_bytes)
from .drafts import verify_drafts
from .pages import (KVPages, kv_cache_compact, kv_cache_copy, kv_pages, kv_pages_fork, kv_pages_release, kv_pages_reserve)

__all__ = ["CapturedAttention", "OvcError", "Prepared", "Repair", "attention", "attention_prepared", "attention_probe",
           "attention_v_repair", "attention_workspace_bytes", "attn_flags", "group_v", "device_status", "flops", "prepare", "prepare_v_repair",
           "prepare_workspace_bytes", "repair_workspace_bytes", "baseline_attention",
           "KVCache", "kv_cache", "kv_cache_read", "kv_cache_write", "paged_attention", "paged_attention_workspace_bytes",
           "KVPages", "kv_cache_compact", "kv_cache_copy", "kv_pages", "kv_pages_fork", "kv_pages_release", "kv_pages_reserve",
           "verify_drafts"]
